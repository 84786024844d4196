"""ctypes binding of libloglinear.so: argument marshalling only.

Every step of the forward and of the decode step runs in the library's CUDA kernels;
this module checks tensor placement / dtype / contiguity, allocates outputs and the
forward's workspace with PyTorch (device memory is PyTorch's job here), passes raw
pointers and sizes to the C ABI on the current CUDA stream, and turns a non-zero status
into an exception.  If the library is missing the import fails loudly: there is no
fallback implementation.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libloglinear.so")

LL_OK, LL_ERR_INVALID, LL_ERR_SHAPE, LL_ERR_DTYPE, LL_ERR_UNSUPPORTED, LL_ERR_CUDA, \
    LL_ERR_WORKSPACE, LL_ERR_ALIGN = range(8)
LL_F32, LL_BF16 = 0, 1
LL_PATH_AUTO, LL_PATH_SIMT, LL_PATH_TC = 0, 1, 2
PATHS = {"auto": LL_PATH_AUTO, "simt": LL_PATH_SIMT, "tc": LL_PATH_TC}

class LLStrides(ctypes.Structure):
    """ll_strides: element strides of the batch, position and head dimensions."""
    _fields_ = [("b", ctypes.c_int64), ("t", ctypes.c_int64), ("h", ctypes.c_int64)]


class LLCache(ctypes.Structure):
    """ll_cache: sizes and arrays of a paged decode cache."""
    _fields_ = [(n, ctypes.c_int64) for n in ("slots", "n_pages", "H", "Hqk", "dk", "dv",
                                              "levels")] + \
        [("dtype", ctypes.c_int)] + \
        [(n, ctypes.c_void_p) for n in ("pages", "page_table", "refcount", "win_k", "win_v",
                                        "win_log_a", "page_log", "page_from", "scratch", "error")]


# Every symbol include/loglinear.h declares, with its ctypes signature.
_i64, _int, _vp, _sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
_sp = ctypes.POINTER(LLStrides)
_cp = ctypes.POINTER(LLCache)
SIGNATURES = {
    "loglinear_version": (_int, []),
    "loglinear_status_string": (ctypes.c_char_p, [_int]),
    "loglinear_last_cuda_error": (ctypes.c_char_p, []),
    "loglinear_fwd_resolve_path": (_int, [_i64, _i64, _int, _int, _int]),
    "loglinear_fwd_workspace_size": (_int, [_i64, _i64, _i64, _i64, _i64, _int, _int, _int,
                                            ctypes.POINTER(_sz)]),
    "loglinear_fwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _i64,
                             _i64, _int, _int, _int, _int, _vp, _sz, _vp]),
    "loglinear_fwd_strided": (_int, [_vp, _sp, _vp, _sp, _vp, _sp, _vp, _vp, _vp, _sp, _i64, _i64,
                                     _i64, _i64, _i64, _i64, _i64, _int, _int, _int, _int, _vp,
                                     _sz, _vp]),
    "loglinear_prefill_with_events": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64,
                                             _i64, _i64, _i64, _i64, _int, _int, _int, _int, _vp,
                                             _sz, _vp, ctypes.POINTER(_vp), _int,
                                             ctypes.POINTER(_int)]),
    "loglinear_fwd_with_events": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64,
                                         _i64, _i64, _i64, _int, _int, _int, _int, _vp, _sz, _vp,
                                         ctypes.POINTER(_vp), _int, ctypes.POINTER(_int)]),
    "loglinear_decode_step": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _i64, _i64, _i64,
                                     _i64, _i64, _i64, _int, _int, _vp]),
    "loglinear_gdn_decode_step": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _i64, _i64,
                                         _i64, _i64, _i64, _i64, _int, _int, _vp]),
    "loglinear_gdn_fwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64,
                                 _i64, _i64, _i64, _int, _int, _vp]),
    "loglinear_gdn_fwd_chunked_workspace_size": (_int, [_i64, _i64, _i64, _i64, _i64,
                                                        ctypes.POINTER(ctypes.c_size_t)]),
    "loglinear_gdn_fwd_chunked": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64,
                                         _i64, _i64, _i64, _i64, _i64, _int, _int, _vp, _sz,
                                         _vp]),
    "loglinear_debug_level_map": (_int, [_i64, _int, _int, _vp, _vp]),
    "loglinear_device_error": (_int, [_vp, ctypes.POINTER(ctypes.c_uint)]),
    "loglinear_fwd_noalloc": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64,
                                     _i64, _i64, _int, _int, _int, _int, _vp]),
    "loglinear_prefill": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64,
                                 _i64, _i64, _int, _int, _int, _int, _vp, _sz, _vp]),
    "loglinear_bwd_workspace_size": (_int, [_i64, _i64, _i64, _i64, _i64, _i64, _i64, _int, _int,
                                            _int, ctypes.POINTER(_sz)]),
    "loglinear_bwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64,
                             _i64, _i64, _i64, _i64, _i64, _int, _int, _int, _vp, _sz, _vp, _sz,
                             _vp]),
    "loglinear_glr_fwd": (_int, [_vp, _sp, _vp, _sp, _vp, _vp, _i64, _vp, _vp, _i64, _i64, _i64,
                                 _int, _int, _int, _int, _vp]),
    "loglinear_glr_bwd": (_int, [_vp, _sp, _vp, _sp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp,
                                 _i64, _i64, _i64, _int, _int, _int, _int, _vp]),
    "loglinear_glr_step": (_int, [_vp, _i64, _vp, _vp, _vp, _vp, _i64, _i64, _int, _int, _int,
                                  _int, _vp]),
    "loglinear_cache_scratch_size": (_int, [_i64, _i64, ctypes.POINTER(_sz)]),
    "loglinear_cache_reserve": (_int, [_cp, _vp, _vp, _i64, _vp]),
    "loglinear_cache_step": (_int, [_cp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _int,
                                    _vp]),
    "loglinear_cache_load": (_int, [_cp, _vp, _i64, _i64, _vp, _i64, _vp, _sp, _vp, _sp, _vp, _sp,
                                    _i64, _vp]),
    "loglinear_cache_store": (_int, [_cp, _vp, _vp, _vp, _i64, _i64, _vp]),
    "loglinear_cache_fork": (_int, [_cp, _vp, _vp, _vp, _i64, _vp]),
    "loglinear_cache_free": (_int, [_cp, _vp, _i64, _vp]),
    "loglinear_cache_compact": (_int, [_cp, _vp, _vp]),
    "loglinear_cache_tree": (_int, [_cp, _vp, _vp, _vp, _vp, _sp, _vp, _sp, _vp, _sp, _vp, _vp, _vp,
                                    _i64, _i64, _i64, _int, _vp]),
    "loglinear_cache_accept": (_int, [_cp, _vp, _vp, _vp, _vp, _sp, _vp, _sp, _vp, _vp, _i64, _i64,
                                      _i64, _vp]),
    "loglinear_tree_verify": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _int,
                                     _vp]),
}


class LoglinearError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = f"{where}: {status_string(status)}"
        if status == LL_ERR_CUDA:
            msg += f" ({_lib.loglinear_last_cuda_error().decode()})"
        super().__init__(msg)
        self.status = status


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = load_library()


def lib() -> ctypes.CDLL:
    return _lib


def status_string(status: int) -> str:
    return _lib.loglinear_status_string(int(status)).decode()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return LL_F32
    if t.dtype == torch.bfloat16:
        return LL_BF16
    raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check_dev(name, t, dtype=None, shape=None, strided=False):
    """Device, dtype and shape checks; contiguity, or with strided=True only a contiguous
    last dimension (the others are passed as strides)."""
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if strided:
        if t.dim() != 4 or (t.shape[-1] > 1 and t.stride(-1) != 1):
            raise ValueError(f"{name} must have a contiguous last dimension")
    elif not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def resolve_path(dk, dv, chunk, in_dtype, path="auto") -> str:
    r = _lib.loglinear_fwd_resolve_path(dk, dv, chunk, in_dtype, PATHS[path])
    if r < 0:
        raise LoglinearError(-r, "loglinear_fwd_resolve_path")
    return {LL_PATH_SIMT: "simt", LL_PATH_TC: "tc"}[r]


def fwd_workspace_size(B, T, H, dk, dv, chunk, in_dtype, path="auto") -> int:
    out = ctypes.c_size_t(0)
    st = _lib.loglinear_fwd_workspace_size(B, T, H, dk, dv, chunk, in_dtype, PATHS[path],
                                           ctypes.byref(out))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_fwd_workspace_size")
    return int(out.value)


def loglinear_fwd(q, k, v, log_a, lam, chunk, out=None, out_dtype=None, workspace=None,
                  path="auto", stream=None):
    """O = (Q K^T ⊙ M^S ⊙ M^H) V through the C ABI (q, k [B,T,Hqk,dk]; v [B,T,H,dv];
    log_a [B,T,H] fp32 or None; lam [B,T,H,L] fp32; head h reads q/k head h // (H/Hqk)).
    q, k, v and out may be strided views with a contiguous last dimension (e.g. slices of
    a fused q/k/v projection); they then go through loglinear_fwd_strided.
    Returns out [B,T,H,dv]."""
    B, T, Hqk, dk = q.shape
    H, dv, L = v.shape[2], v.shape[-1], lam.shape[-1]
    _check_dev("q", q, shape=(B, T, Hqk, dk), strided=True)
    _check_dev("k", k, q.dtype, (B, T, Hqk, dk), strided=True)
    _check_dev("v", v, q.dtype, (B, T, H, dv), strided=True)
    _check_dev("log_a", log_a, torch.float32, (B, T, H))
    _check_dev("lam", lam, torch.float32, (B, T, H, L))
    in_dt = _dtype_code(q)
    if out is None:
        out = torch.empty(B, T, H, dv, device=q.device, dtype=out_dtype or q.dtype)
    _check_dev("out", out, shape=(B, T, H, dv), strided=True)
    ws_bytes = fwd_workspace_size(B, T, H, dk, dv, chunk, in_dt, path)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), device=q.device, dtype=torch.uint8)
    _check_dev("workspace", workspace, torch.uint8)
    if all(x.is_contiguous() for x in (q, k, v, out)):
        st = _lib.loglinear_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_a), _ptr(lam), _ptr(out),
                                B, T, H, Hqk, dk, dv, L, chunk, in_dt, _dtype_code(out),
                                PATHS[path], _ptr(workspace), workspace.numel(), _stream(stream))
    else:
        sd = [ctypes.byref(LLStrides(*x.stride()[:3])) for x in (q, k, v, out)]
        st = _lib.loglinear_fwd_strided(_ptr(q), sd[0], _ptr(k), sd[1], _ptr(v), sd[2],
                                        _ptr(log_a), _ptr(lam), _ptr(out), sd[3], B, T, H, Hqk, dk,
                                        dv, L, chunk, in_dt, _dtype_code(out), PATHS[path],
                                        _ptr(workspace), workspace.numel(), _stream(stream))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_fwd")
    return out


def loglinear_fwd_with_events(q, k, v, log_a, lam, chunk, events, out, workspace, path="auto",
                              stream=None):
    """loglinear_fwd plus torch.cuda.Event records between its kernels (events are
    created with enable_timing=True by the caller).  Returns the number of kernels."""
    B, T, Hqk, dk = q.shape
    H, dv, L = v.shape[2], v.shape[-1], lam.shape[-1]
    st_ = stream if stream is not None else torch.cuda.current_stream()
    for e in events:          # torch creates the CUDA event lazily, on its first record
        if not e.cuda_event:
            e.record(st_)
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    nk = ctypes.c_int(0)
    st = _lib.loglinear_fwd_with_events(_ptr(q), _ptr(k), _ptr(v), _ptr(log_a), _ptr(lam),
                                        _ptr(out), B, T, H, Hqk, dk, dv, L, chunk, _dtype_code(q),
                                        _dtype_code(out), PATHS[path], _ptr(workspace),
                                        workspace.numel(), _stream(stream), arr, len(events),
                                        ctypes.byref(nk))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_fwd_with_events")
    return nk.value


def loglinear_decode_step(state, q, k, v, log_a, lam, t, out=None, out_dtype=None, stream=None):
    """One lssb decode step at position t; updates state [B,H,L,dk,dv] (fp32) in place
    and returns out [B,H,dv].  q, k [B,Hqk,dk] (head h reads q/k head h // (H/Hqk))."""
    B, H, L, dk, dv = state.shape
    Hqk = q.shape[1]
    _check_dev("state", state, torch.float32)
    _check_dev("q", q, shape=(B, Hqk, dk))
    _check_dev("k", k, q.dtype, (B, Hqk, dk))
    _check_dev("v", v, q.dtype, (B, H, dv))
    _check_dev("log_a", log_a, torch.float32, (B, H))
    _check_dev("lam", lam, torch.float32, (B, H, L))
    if out is None:
        out = torch.empty(B, H, dv, device=q.device, dtype=out_dtype or q.dtype)
    _check_dev("out", out, shape=(B, H, dv))
    st = _lib.loglinear_decode_step(_ptr(state), _ptr(q), _ptr(k), _ptr(v), _ptr(log_a),
                                    _ptr(lam), int(t), _ptr(out), B, H, Hqk, dk, dv, L, _dtype_code(q),
                                    _dtype_code(out), _stream(stream))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_decode_step")
    return out


def loglinear_gdn_decode_step(state, q, k, v, log_a, beta, lam, t, out=None, out_dtype=None,
                              stream=None):
    """One Log-Linear Gated DeltaNet decode step at position t; updates state [B,H,L,dk,dv]
    (fp32) in place and returns out [B,H,dv].  q, k [B,Hqk,dk]; beta [B,H] fp32."""
    B, H, L, dk, dv = state.shape
    Hqk = q.shape[1]
    _check_dev("state", state, torch.float32)
    _check_dev("q", q, shape=(B, Hqk, dk))
    _check_dev("k", k, q.dtype, (B, Hqk, dk))
    _check_dev("v", v, q.dtype, (B, H, dv))
    _check_dev("log_a", log_a, torch.float32, (B, H))
    _check_dev("beta", beta, torch.float32, (B, H))
    _check_dev("lam", lam, torch.float32, (B, H, L))
    if out is None:
        out = torch.empty(B, H, dv, device=q.device, dtype=out_dtype or q.dtype)
    _check_dev("out", out, shape=(B, H, dv))
    st = _lib.loglinear_gdn_decode_step(_ptr(state), _ptr(q), _ptr(k), _ptr(v), _ptr(log_a),
                                        _ptr(beta), _ptr(lam), int(t), _ptr(out), B, H, Hqk, dk,
                                        dv, L, _dtype_code(q), _dtype_code(out), _stream(stream))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_gdn_decode_step")
    return out


def loglinear_gdn_fwd(q, k, v, log_a, beta, lam, out=None, out_dtype=None, state=None,
                      stream=None):
    """Log-Linear Gated DeltaNet over a whole sequence (recurrent form).  q, k [B,T,Hqk,dk];
    v [B,T,H,dv]; log_a [B,T,H] fp32 or None; beta [B,T,H] fp32; lam [B,T,H,L] fp32.
    Returns out [B,T,H,dv]; when `state` ([B,H,L,dk,dv] fp32) is given it receives the
    per-level state after position T-1."""
    B, T, Hqk, dk = q.shape
    H, dv, L = v.shape[2], v.shape[-1], lam.shape[-1]
    _check_dev("q", q)
    _check_dev("k", k, q.dtype, (B, T, Hqk, dk))
    _check_dev("v", v, q.dtype, (B, T, H, dv))
    _check_dev("log_a", log_a, torch.float32, (B, T, H))
    _check_dev("beta", beta, torch.float32, (B, T, H))
    _check_dev("lam", lam, torch.float32, (B, T, H, L))
    if state is not None:
        _check_dev("state", state, torch.float32, (B, H, L, dk, dv))
    if out is None:
        out = torch.empty(B, T, H, dv, device=q.device, dtype=out_dtype or q.dtype)
    _check_dev("out", out, shape=(B, T, H, dv))
    st = _lib.loglinear_gdn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_a), _ptr(beta), _ptr(lam),
                                _ptr(out), _ptr(state), B, T, H, Hqk, dk, dv, L, _dtype_code(q),
                                _dtype_code(out), _stream(stream))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_gdn_fwd")
    return out


def gdn_fwd_chunked_workspace_size(B, T, H, dk, dv) -> int:
    out = ctypes.c_size_t(0)
    st = _lib.loglinear_gdn_fwd_chunked_workspace_size(B, T, H, dk, dv, ctypes.byref(out))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_gdn_fwd_chunked_workspace_size")
    return int(out.value)


def loglinear_gdn_fwd_chunked(q, k, v, log_a, beta, lam, out=None, out_dtype=None,
                              workspace=None, state=None, stream=None):
    """Log-Linear Gated DeltaNet over a whole sequence in chunks of 64 tokens (same inputs and
    output as loglinear_gdn_fwd; `state`, [B,H,L,dk,dv] fp32, receives the decode state after
    T-1 when given).  The workspace is allocated with torch when not given."""
    B, T, Hqk, dk = q.shape
    H, dv, L = v.shape[2], v.shape[-1], lam.shape[-1]
    _check_dev("q", q)
    _check_dev("k", k, q.dtype, (B, T, Hqk, dk))
    _check_dev("v", v, q.dtype, (B, T, H, dv))
    _check_dev("log_a", log_a, torch.float32, (B, T, H))
    _check_dev("beta", beta, torch.float32, (B, T, H))
    _check_dev("lam", lam, torch.float32, (B, T, H, L))
    if state is not None:
        _check_dev("state", state, torch.float32, (B, H, L, dk, dv))
    if out is None:
        out = torch.empty(B, T, H, dv, device=q.device, dtype=out_dtype or q.dtype)
    _check_dev("out", out, shape=(B, T, H, dv))
    sz = ctypes.c_size_t(0)
    st = _lib.loglinear_gdn_fwd_chunked_workspace_size(B, T, H, dk, dv, ctypes.byref(sz))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_gdn_fwd_chunked_workspace_size")
    if workspace is None:
        workspace = torch.empty(max(sz.value, 1), device=q.device, dtype=torch.uint8)
    st = _lib.loglinear_gdn_fwd_chunked(_ptr(q), _ptr(k), _ptr(v), _ptr(log_a), _ptr(beta),
                                        _ptr(lam), _ptr(out), _ptr(state), B, T, H, Hqk, dk, dv,
                                        L,
                                        _dtype_code(q), _dtype_code(out), _ptr(workspace),
                                        workspace.numel(), _stream(stream))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_gdn_fwd_chunked")
    return out


def loglinear_prefill_with_events(q, k, v, log_a, lam, chunk, events, out, state, workspace,
                                  path="auto", stream=None):
    """loglinear_prefill plus torch.cuda.Event records between its kernels (the last
    kernel forms the decode state).  Returns the number of kernels."""
    B, T, Hqk, dk = q.shape
    H, dv, L = v.shape[2], v.shape[-1], lam.shape[-1]
    st_ = stream if stream is not None else torch.cuda.current_stream()
    for e in events:          # torch creates the CUDA event lazily, on its first record
        if not e.cuda_event:
            e.record(st_)
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    nk = ctypes.c_int(0)
    st = _lib.loglinear_prefill_with_events(_ptr(q), _ptr(k), _ptr(v), _ptr(log_a), _ptr(lam),
                                            _ptr(out), _ptr(state), B, T, H, Hqk, dk, dv, L,
                                            chunk, _dtype_code(q), _dtype_code(out), PATHS[path],
                                            _ptr(workspace), workspace.numel(), _stream(stream),
                                            arr, len(events), ctypes.byref(nk))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_prefill_with_events")
    return nk.value


def loglinear_prefill(q, k, v, log_a, lam, chunk, out=None, state=None, out_dtype=None,
                      workspace=None, path="auto", stream=None):
    """loglinear_fwd over the prompt plus the per-level decode state at its last position
    (fp32 [B, H, L, dk, dv]), ready for loglinear_decode_step at t = T.
    Returns (out, state).  q/k heads as in loglinear_fwd."""
    B, T, Hqk, dk = q.shape
    H, dv, L = v.shape[2], v.shape[-1], lam.shape[-1]
    _check_dev("q", q, shape=(B, T, Hqk, dk))
    _check_dev("k", k, q.dtype, (B, T, Hqk, dk))
    _check_dev("v", v, q.dtype, (B, T, H, dv))
    _check_dev("log_a", log_a, torch.float32, (B, T, H))
    _check_dev("lam", lam, torch.float32, (B, T, H, L))
    in_dt = _dtype_code(q)
    if out is None:
        out = torch.empty(B, T, H, dv, device=q.device, dtype=out_dtype or q.dtype)
    if state is None:
        state = torch.empty(B, H, L, dk, dv, device=q.device, dtype=torch.float32)
    _check_dev("out", out, shape=(B, T, H, dv))
    _check_dev("state", state, torch.float32, (B, H, L, dk, dv))
    ws_bytes = fwd_workspace_size(B, T, H, dk, dv, chunk, in_dt, path) if T > 0 else 0
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), device=q.device, dtype=torch.uint8)
    _check_dev("workspace", workspace, torch.uint8)
    st = _lib.loglinear_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(log_a), _ptr(lam), _ptr(out),
                                _ptr(state), B, T, H, Hqk, dk, dv, L, chunk, in_dt, _dtype_code(out),
                                PATHS[path], _ptr(workspace), workspace.numel(), _stream(stream))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_prefill")
    return out, state


def loglinear_fwd_noalloc(q, k, v, log_a, lam, chunk, out, path="auto", stream=None):
    """loglinear_fwd without a workspace, for callers that cannot allocate device memory:
    the scratch is the library's fixed device array (see include/loglinear.h).  `out` is
    caller-provided; nothing is allocated here either."""
    B, T, Hqk, dk = q.shape
    H, dv, L = v.shape[2], v.shape[-1], lam.shape[-1]
    for name, t in (("q", q), ("k", k), ("v", v), ("log_a", log_a), ("lam", lam), ("out", out)):
        _check_dev(name, t)
    st = _lib.loglinear_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(log_a), _ptr(lam), _ptr(out),
                                    B, T, H, Hqk, dk, dv, L, chunk, _dtype_code(q), _dtype_code(out),
                                    PATHS[path], _stream(stream))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_fwd_noalloc")
    return out


def bwd_workspace_size(B, T, H, Hqk, dk, dv, L, in_dtype, grad_dtype, path="auto") -> int:
    out = ctypes.c_size_t(0)
    st = _lib.loglinear_bwd_workspace_size(B, T, H, Hqk, dk, dv, L, in_dtype, grad_dtype,
                                           PATHS[path], ctypes.byref(out))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_bwd_workspace_size")
    return int(out.value)


def loglinear_bwd(q, k, v, log_a, lam, dout, workspace=None, path="auto", fwd_workspace=None,
                  stream=None):
    """Gradients of sum(dout ⊙ O) for O = loglinear_fwd(q, k, v, log_a, lam): returns
    (dq, dk, dv, dlog_a, dlam); dq, dk, dv in dout's dtype, dlog_a (None without decay)
    and dlam fp32.  path: "tc" computes dq and dlam on the tensor cores (bf16, d_k = 128,
    d_v in {64, 128}), "simt" everything on CUDA cores, "auto" the tensor cores if they
    apply.  fwd_workspace: the workspace of a tensor-core loglinear_fwd over the same
    inputs, whose block states are then read instead of recomputed."""
    B, T, Hqk, dk = q.shape
    H, dv, L = v.shape[2], v.shape[-1], lam.shape[-1]
    _check_dev("q", q, shape=(B, T, Hqk, dk))
    _check_dev("k", k, q.dtype, (B, T, Hqk, dk))
    _check_dev("v", v, q.dtype, (B, T, H, dv))
    _check_dev("log_a", log_a, torch.float32, (B, T, H))
    _check_dev("lam", lam, torch.float32, (B, T, H, L))
    _check_dev("dout", dout, shape=(B, T, H, dv))
    in_dt, g_dt = _dtype_code(q), _dtype_code(dout)
    dq = torch.empty_like(q, dtype=dout.dtype)
    dk_ = torch.empty_like(k, dtype=dout.dtype)
    dv_ = torch.empty_like(v, dtype=dout.dtype)
    dla = None if log_a is None else torch.empty_like(log_a)
    dlam = torch.empty_like(lam)
    ws_bytes = bwd_workspace_size(B, T, H, Hqk, dk, dv, L, in_dt, g_dt, path)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), device=q.device, dtype=torch.uint8)
    _check_dev("workspace", workspace, torch.uint8)
    if fwd_workspace is not None:
        _check_dev("fwd_workspace", fwd_workspace, torch.uint8)
    st = _lib.loglinear_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_a), _ptr(lam), _ptr(dout),
                            _ptr(dq), _ptr(dk_), _ptr(dv_), _ptr(dla), _ptr(dlam), B, T, H, Hqk,
                            dk, dv, L, in_dt, g_dt, PATHS[path], _ptr(fwd_workspace),
                            0 if fwd_workspace is None else fwd_workspace.numel(),
                            _ptr(workspace), workspace.numel(), _stream(stream))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_bwd")
    return dq, dk_, dv_, dla, dlam


def device_error(stream=None) -> int:
    """Reads and clears the tensor-core path's device error word (0 = no bounded wait
    ran out of time).  Synchronises the stream."""
    flags = ctypes.c_uint(0)
    st = _lib.loglinear_device_error(_stream(stream), ctypes.byref(flags))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_device_error")
    return int(flags.value)


def debug_level_map(T, chunk, path="auto", stream=None):
    """[T, T] int8 map of the level the forward's decomposition gives each (t, s)."""
    out = torch.empty(T, T, device="cuda", dtype=torch.int8)
    st = _lib.loglinear_debug_level_map(T, chunk, PATHS[path], _ptr(out), _stream(stream))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_debug_level_map")
    return out


# ---------------------------------------------------------------- gated linear recurrence

GLR_SCALES = {"none": 0, "one_minus": 1, "sqrt": 2}


def _here(name, t, dtype=None, shape=None):
    """_check_dev for one tensor of a call whose kernels run on the current device."""
    if t is None:
        return
    _check_dev(name, t, dtype, shape)
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, not on the current device")


def _at(name, t, dtype, shape, dev):
    """The address of a contiguous tensor on device `dev`, the current one (None: no tensor).
    A step's calls take about as long on the host as on the GPU: one test where all is well."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _here(name, t, dtype, shape)
    raise ValueError(f"{name} is not as expected")


def _current_device_of(name, t):
    """The current device, which has to be t's."""
    dev = t.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        raise ValueError(f"{name} must be a CUDA tensor on the current device, got {t.device}")
    return dev


def _raw_stream(stream, dev):
    """The stream's handle (None: the current one)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)  # current_stream() takes 3 us
    return stream.cuda_stream


def _token_strides(name, t, shape, dtype=None, features=True):
    """An input with strided batch, position (and head) dimensions, its features (if it has
    any) contiguous: its strides, or None when dense."""
    if t is None:
        return None
    if not t.is_cuda or t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} must be a CUDA tensor on the current device")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.is_contiguous():
        return None
    if features and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have a contiguous last dimension")
    s = t.stride()[:-1] if features else t.stride()
    return ctypes.byref(LLStrides(s[0], s[1], s[2] if len(s) > 2 else 0))


def _empty(stream, *shape, **kw):
    """torch.empty owned by the stream the kernels run on, so that memory freed after the call
    is only reused behind them."""
    if stream is None:
        return torch.empty(*shape, **kw)
    with torch.cuda.stream(stream):
        return torch.empty(*shape, **kw)


def _glr_sequences(cu_seqlens, B):
    if cu_seqlens is None:
        return B
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must have shape [N + 1]")
    return cu_seqlens.numel() - 1


def _glr_input(name, t, shape, dev):
    """Address and strides (None: dense) of an input."""
    if t is None:
        return None, None
    if t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr(), None
    return t.data_ptr(), _token_strides(name, t, shape)


def loglinear_glr_fwd(x, log_a, h0=None, cu_seqlens=None, scale="none", out=None, out_dtype=None,
                      state=None, stream=None):
    """Gated linear recurrence h_t = exp(log_a_t) h_{t-1} + b_t x_t per channel; x, log_a
    [B,T,D] (may be views with contiguous channels), log_a fp32 or x's dtype; scale: b = 1
    ("none"), 1 - a ("one_minus") or sqrt(1 - a^2) ("sqrt").  cu_seqlens int32 [N+1] packs N
    sequences into B = 1; rows of out that none of them has are not written.  h0, state: [N,D] fp32
    first states and, when given, where the last ones go.  Returns out [B,T,D]."""
    shape = B, T, D = x.shape
    dev = _current_device_of("x", x)
    xp, xs = _glr_input("x", x, shape, dev)
    lp, ls = _glr_input("log_a", log_a, shape, dev)
    N = _glr_sequences(cu_seqlens, B)
    if out is None:
        out = _empty(stream, B, T, D, device=x.device, dtype=out_dtype or x.dtype)
    st = _lib.loglinear_glr_fwd(
        xp, xs, lp, ls, _at("h0", h0, torch.float32, (N, D), dev),
        _at("cu_seqlens", cu_seqlens, torch.int32, (N + 1,), dev), N,
        _at("out", out, out.dtype, shape, dev), _at("state", state, torch.float32, (N, D), dev), B,
        T, D, _dtype_code(x), _dtype_code(log_a), _dtype_code(out), GLR_SCALES[scale],
        _raw_stream(stream, dev))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_glr_fwd")
    return out


def loglinear_glr_bwd(x, log_a, out, dout, h0=None, cu_seqlens=None, scale="none", dstate=None,
                      stream=None, dx=None, dlog_a=None, dh0=None):
    """Gradients of loglinear_glr_fwd: out is its result, dout (same dtype) the gradient of it,
    dstate [N,D] fp32 that of the last states.  Returns (dx, dlog_a, dh0); dx in dout's dtype,
    dlog_a in log_a's, dh0 fp32 (None without h0; dh0 may be dstate itself).  x may be None with
    scale "none".  Rows of dx and dlog_a that no sequence of cu_seqlens has are not written: give
    both, zeroed once, where a padded batch's gradients go on as a whole."""
    shape = B, T, D = log_a.shape
    dev = _current_device_of("log_a", log_a)
    xp, xs = _glr_input("x", x, shape, dev)
    lp, ls = _glr_input("log_a", log_a, shape, dev)
    N = _glr_sequences(cu_seqlens, B)
    op = _at("out", out, out.dtype, shape, dev)
    gp = _at("dout", dout, out.dtype, shape, dev)
    hp = _at("h0", h0, torch.float32, (N, D), dev)
    sp = _at("dstate", dstate, torch.float32, (N, D), dev)
    cp = _at("cu_seqlens", cu_seqlens, torch.int32, (N + 1,), dev)
    if dx is None:
        dx = _empty(stream, B, T, D, device=out.device, dtype=dout.dtype)
    if dlog_a is None:
        dlog_a = _empty(stream, B, T, D, device=out.device, dtype=log_a.dtype)
    if dh0 is None and h0 is not None:
        dh0 = _empty(stream, N, D, device=out.device, dtype=torch.float32)
    gate = _dtype_code(log_a)
    st = _lib.loglinear_glr_bwd(xp, xs, lp, ls, hp, cp, N, op, gp, sp,
                                _at("dx", dx, dout.dtype, shape, dev),
                                _at("dlog_a", dlog_a, log_a.dtype, shape, dev),
                                _at("dh0", dh0, torch.float32, (N, D), dev), B, T, D,
                                gate if x is None else _dtype_code(x), gate, _dtype_code(out),
                                GLR_SCALES[scale], _raw_stream(stream, dev))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_glr_bwd")
    return dx, dlog_a, dh0


def loglinear_glr_step(state, x, log_a, slots=None, scale="none", out=None, out_dtype=None,
                       stream=None):
    """One token of the recurrence per row: state [S,D] fp32 is updated in place at slots (int32
    [B], -1 leaves the row out; None: row b is slot b).  x, log_a [B,D].  Returns out [B,D]."""
    B, D = x.shape
    dev = _current_device_of("x", x)
    if state.dim() != 2 or state.shape[1] != D:
        raise ValueError(f"state has shape {tuple(state.shape)}, expected (S, {D})")
    if out is None:
        out = _empty(stream, B, D, device=x.device, dtype=out_dtype or x.dtype)
    st = _lib.loglinear_glr_step(
        _at("state", state, torch.float32, state.shape, dev), state.shape[0],
        _at("slots", slots, torch.int32, (B,), dev), _at("x", x, x.dtype, (B, D), dev),
        _at("log_a", log_a, log_a.dtype, (B, D), dev), _at("out", out, out.dtype, (B, D), dev), B, D,
        _dtype_code(x), _dtype_code(log_a), _dtype_code(out), GLR_SCALES[scale],
        _raw_stream(stream, dev))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_glr_step")
    return out


# ---------------------------------------------------------------- paged decode cache

CACHE_BLOCK = 64  # positions of a block (LL_CACHE_BLOCK)
CACHE_ERR_SLOT, CACHE_ERR_POSITION, CACHE_ERR_PAGES, CACHE_ERR_MISSING, CACHE_ERR_WAIT = 1, 2, 4, 8, 16
CACHE_ERR_TREE = 32
TREE_MAX = 64  # nodes of a tree (LL_TREE_MAX)


class LogLinearCache:
    """A paged decode cache over tensors of the caller's (see ll_cache in include/loglinear.h):
    pages [n_pages,H,dk,dv] fp32, page_table [slots,M] int32 (-1: none), refcount [n_pages]
    int32, win_k [slots,Hqk,64,dk] and win_v [slots,H,64,dv] (fp32 or bf16), win_log_a
    [slots,H,64], page_log [slots,2,M,H] fp32 and page_from [slots,2] int32.  `empty` makes
    them.  Calls on one cache have to be ordered: one stream, or events between streams."""

    def __init__(self, pages, page_table, refcount, win_k, win_v, win_log_a, page_log, page_from):
        P, H, dk, dv = pages.shape
        S, M = page_table.shape
        Hqk = win_k.shape[1]
        _here("pages", pages, torch.float32)
        _here("page_table", page_table, torch.int32)
        _here("refcount", refcount, torch.int32, (P,))
        _here("win_k", win_k, None, (S, Hqk, CACHE_BLOCK, dk))
        _here("win_v", win_v, win_k.dtype, (S, H, CACHE_BLOCK, dv))
        _here("win_log_a", win_log_a, torch.float32, (S, H, CACHE_BLOCK))
        _here("page_log", page_log, torch.float32, (S, 2, M, H))
        _here("page_from", page_from, torch.int32, (S, 2))
        self.pages, self.page_table, self.refcount = pages, page_table, refcount
        self.win_k, self.win_v, self.win_log_a = win_k, win_v, win_log_a
        self.page_log, self.page_from = page_log, page_from
        self.slots, self.levels, self.heads, self.qk_heads = S, M, H, Hqk
        self.dk, self.dv, self.dtype, self.device = dk, dv, win_k.dtype, pages.device
        size = ctypes.c_size_t(0)
        st = _lib.loglinear_cache_scratch_size(S, P, ctypes.byref(size))
        if st != LL_OK:
            raise LoglinearError(st, "loglinear_cache_scratch_size")
        self.scratch = torch.empty(size.value, device=pages.device, dtype=torch.uint8)
        self.error_word = torch.zeros(1, device=pages.device, dtype=torch.int32)
        self._struct = LLCache(S, P, H, Hqk, dk, dv, M, _dtype_code(win_k),
                               *(t.data_ptr() for t in (pages, page_table, refcount, win_k, win_v,
                                                        win_log_a, page_log, page_from,
                                                        self.scratch, self.error_word)))
        self._ref = ctypes.byref(self._struct)

    @classmethod
    def empty(cls, slots, n_pages, H, dk, dv, levels, Hqk=None, dtype=torch.bfloat16,
              device="cuda"):
        """A cache that holds nothing: `slots` sequences of fewer than 64 * 2^levels positions
        over a pool of n_pages pages."""
        Hqk = H if Hqk is None else Hqk

        def new(*shape, dt=torch.float32):
            return torch.zeros(*shape, device=device, dtype=dt)

        i32 = torch.int32
        return cls(pages=torch.empty(n_pages, H, dk, dv, device=device),
                   page_table=torch.full((slots, levels), -1, device=device, dtype=i32),
                   refcount=new(n_pages, dt=i32), win_k=new(slots, Hqk, CACHE_BLOCK, dk, dt=dtype),
                   win_v=new(slots, H, CACHE_BLOCK, dv, dt=dtype),
                   win_log_a=new(slots, H, CACHE_BLOCK), page_log=new(slots, 2, levels, H),
                   page_from=new(slots, 2, dt=i32))

    def error(self, stream=None) -> int:
        """Reads and clears the cache's error word (CACHE_ERR_* bits) behind the calls made so far on
        `stream` (None: the current one), which it synchronises.  Calls that went to another
        stream are only seen once that one is ordered before it."""
        with torch.cuda.stream(stream):  # (None: no change)
            bits = int(self.error_word.item())
            if bits:
                self.error_word.zero_()
        return bits

    def _dev(self):
        """The cache's device, which has to be the current one."""
        dev = self.device.index
        if torch.cuda.current_device() != dev:
            raise ValueError(f"the cache is on {self.device}, not on the current device")
        return dev


def loglinear_cache_reserve(cache, slots, pos, stream=None):
    """The page reservation that goes before a loglinear_cache_step at the same slots and
    positions (int32 [n] each): pages no longer live are given up, and slots at a block's last
    position take the page it is folded into."""
    dev, n = cache._dev(), slots.numel()
    st = _lib.loglinear_cache_reserve(cache._ref, _at("slots", slots, torch.int32, (n,), dev),
                                      _at("pos", pos, torch.int32, (n,), dev), n,
                                      _raw_stream(stream, dev))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_cache_reserve")


def loglinear_cache_step(cache, slots, pos, q, k, v, log_a, lam, out=None, out_dtype=None,
                         stream=None):
    """One decode step for n rows, row i being slot slots[i] at position pos[i].  q, k [n,Hqk,dk],
    v [n,H,dv] in the cache's dtype; log_a [n,H] fp32 or None; lam [n,H,L] fp32, L >= levels + 7.
    Rows with slot -1 are left out (their out is not written).  A slot may go back to earlier
    positions of its block until it has been called for in the next one (drafts that cross a block's
    end: on a fork).  Returns out [n,H,dv]."""
    dev, n, L = cache._dev(), slots.numel(), lam.shape[-1]
    dt, H, qk = cache.dtype, cache.heads, (n, cache.qk_heads, cache.dk)
    if out is None:
        out = _empty(stream, n, H, cache.dv, device=q.device, dtype=out_dtype or q.dtype)
    st = _lib.loglinear_cache_step(
        cache._ref, _at("slots", slots, torch.int32, (n,), dev), _at("pos", pos, torch.int32, (n,), dev),
        _at("q", q, dt, qk, dev), _at("k", k, dt, qk, dev), _at("v", v, dt, (n, H, cache.dv), dev),
        _at("log_a", log_a, torch.float32, (n, H), dev), _at("lam", lam, torch.float32, (n, H, L), dev),
        _at("out", out, out.dtype, (n, H, cache.dv), dev), n, L, _dtype_code(out),
        _raw_stream(stream, dev))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_cache_step")
    return out


def loglinear_cache_load(cache, slots, T, state, k, v, log_a, stream=None):
    """Puts n prompts of T positions into slots (int32 [n]), which give up what they held.  state
    [n,H,L,dk,dv] fp32 as loglinear_prefill returns it; k [n,Tk,Hqk,dk], v [n,Tk,H,dv], log_a
    [n,Tk,H] or None: the prompt's last Tk >= T mod 64 tokens (views such as k[:, -64:] do)."""
    dev, n = cache._dev(), slots.numel()
    L, Tk = state.shape[2], k.shape[1]
    sk = _token_strides("k", k, (n, Tk, cache.qk_heads, cache.dk), cache.dtype)
    sv = _token_strides("v", v, (n, Tk, cache.heads, cache.dv), cache.dtype)
    sa = _token_strides("log_a", log_a, (n, Tk, cache.heads), torch.float32, features=False)
    st = _lib.loglinear_cache_load(
        cache._ref, _at("slots", slots, torch.int32, (n,), dev), n, T,
        _at("state", state, torch.float32, (n, cache.heads, L, cache.dk, cache.dv), dev), L,
        k.data_ptr(), sk, v.data_ptr(), sv, _ptr(log_a), sa, Tk, _raw_stream(stream, dev))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_cache_load")


def loglinear_cache_store(cache, slots, pos, state=None, stream=None):
    """Dense states [n,H,L,dk,dv] fp32 (L >= levels + 7) of slots that hold pos positions, from
    which loglinear_decode_step goes on at t = pos.  Returns state."""
    dev, n = cache._dev(), slots.numel()
    if state is None:
        state = _empty(stream, n, cache.heads, cache.levels + 7, cache.dk, cache.dv,
                       device=cache.device)
    L = state.shape[2]
    st = _lib.loglinear_cache_store(
        cache._ref, _at("slots", slots, torch.int32, (n,), dev), _at("pos", pos, torch.int32, (n,), dev),
        _at("state", state, torch.float32, (n, cache.heads, L, cache.dk, cache.dv), dev), n, L,
        _raw_stream(stream, dev))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_cache_store")
    return state


def loglinear_cache_fork(cache, src, dst, pos, stream=None):
    """Slot dst[i] becomes a copy of slot src[i], which holds pos[i] positions (int32 [n] each):
    pages are shared, the block's tokens copied."""
    dev, n = cache._dev(), src.numel()
    st = _lib.loglinear_cache_fork(
        cache._ref, _at("src", src, torch.int32, (n,), dev), _at("dst", dst, torch.int32, (n,), dev),
        _at("pos", pos, torch.int32, (n,), dev), n, _raw_stream(stream, dev))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_cache_fork")


def loglinear_cache_free(cache, slots, stream=None):
    """The slots (int32 [n]) give up their pages."""
    dev, n = cache._dev(), slots.numel()
    st = _lib.loglinear_cache_free(cache._ref, _at("slots", slots, torch.int32, (n,), dev), n,
                                   _raw_stream(stream, dev))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_cache_free")


def loglinear_cache_compact(cache, live=None, stream=None):
    """Moves pages so that those in use are the lowest.  Returns their number, int32 [1] on the
    device."""
    dev = cache._dev()
    if live is None:
        live = _empty(stream, 1, device=cache.device, dtype=torch.int32)
    st = _lib.loglinear_cache_compact(cache._ref, _at("live", live, torch.int32, (1,), dev),
                                      _raw_stream(stream, dev))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_cache_compact")
    return live


# ---------------------------------------------------------------- speculative decoding

def _drafts(name, t, shape, dtype, dev):
    """Address and strides (None: dense) of a tree's q, k or v, views with contiguous features."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr(), None
    return t.data_ptr(), _token_strides(name, t, shape, dtype)


def loglinear_cache_tree(cache, slots, pos, parents, q, k, v, log_a, lam, out=None, out_dtype=None,
                         stream=None):
    """The decode step's attention for trees of N <= 64 drafted tokens: row i's nodes follow the
    pos[i] positions of slot slots[i] (int32 [n]; -1 leaves the row out) and their own parents.
    parents [n,N] int32: an earlier node, -1 (the context) or -2 (the node is left out; its out is not
    written).  q, k [n,N,Hqk,dk], v [n,N,H,dv] in the cache's dtype (may be views with
    contiguous features); log_a [n,N,H] fp32 or None; lam [n,N,H,L] fp32, L >= levels + 7.  The cache
    is not changed.  Returns out [n,N,H,dv]."""
    dev, n, L = cache._dev(), slots.numel(), lam.shape[-1]
    N = q.shape[1]
    dt, H, qk, vs = cache.dtype, cache.heads, (n, N, cache.qk_heads, cache.dk), (n, N, cache.heads, cache.dv)
    qp, sq = _drafts("q", q, qk, dt, dev)
    kp, sk = _drafts("k", k, qk, dt, dev)
    vp, sv = _drafts("v", v, vs, dt, dev)
    if out is None:
        out = _empty(stream, *vs, device=q.device, dtype=out_dtype or q.dtype)
    st = _lib.loglinear_cache_tree(
        cache._ref, _at("slots", slots, torch.int32, (n,), dev), _at("pos", pos, torch.int32, (n,), dev),
        _at("parents", parents, torch.int32, (n, N), dev), qp, sq, kp, sk, vp, sv,
        _at("log_a", log_a, torch.float32, (n, N, H), dev),
        _at("lam", lam, torch.float32, (n, N, H, L), dev), _at("out", out, out.dtype, vs, dev), n, N, L,
        _dtype_code(out), _raw_stream(stream, dev))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_cache_tree")
    return out


def loglinear_tree_verify(parents, tokens, probs, u, draft=None, path=None, count=None, token=None,
                          stream=None):
    """Which drafts of a tree stand, by speculative sampling from given random numbers: distributed as
    the target's tokens where the rows of probs (and draft) sum to 1.  parents, tokens [n,N] int32
    (node 0: the pending token; a row whose node 0 is -2 is padding); probs [n,N,V] fp32 or bf16: the
    target's distribution after each node; u [n,N] fp32 in [0,1), u[:,0] for the next token; draft
    [n,N,V] in probs' dtype: the distribution that each node's children were drawn from, or None for
    drafts that were given.  Returns (path [n,N] int32: node 0, the accepted nodes, -1 behind them;
    count [n] int32; token [n] int32: the next pending token), allocated where they are not given."""
    dev = _current_device_of("probs", probs)
    if probs.dim() != 3:
        raise ValueError(f"probs has shape {tuple(probs.shape)}, expected (n, N, V)")
    n, N, V = probs.shape
    i32 = torch.int32
    if path is None:
        path = _empty(stream, n, N, device=probs.device, dtype=i32)
    if count is None:
        count = _empty(stream, n, device=probs.device, dtype=i32)
    if token is None:
        token = _empty(stream, n, device=probs.device, dtype=i32)
    st = _lib.loglinear_tree_verify(
        _at("parents", parents, i32, (n, N), dev), _at("tokens", tokens, i32, (n, N), dev),
        _at("probs", probs, probs.dtype, (n, N, V), dev), _at("draft", draft, probs.dtype, (n, N, V), dev),
        _at("u", u, torch.float32, (n, N), dev), _at("path", path, i32, (n, N), dev),
        _at("count", count, i32, (n,), dev), _at("token", token, i32, (n,), dev), n, N, V,
        _dtype_code(probs), _raw_stream(stream, dev))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_tree_verify")
    return path, count, token


def loglinear_cache_accept(cache, slots, pos, path, k, v, log_a, new_pos=None, stream=None):
    """The nodes of path ([n,D] int32, up to the first -1) join their slots from pos on, as
    loglinear_cache_step would have put them there, reservation and fold included; k, v, log_a are
    those of loglinear_cache_tree.  Returns new_pos [n] int32, pos + the path's length (rows that are
    left out keep what it held: give one that is initialised where that matters)."""
    dev, n = cache._dev(), slots.numel()
    N, D = k.shape[1], path.shape[-1]
    kp, sk = _drafts("k", k, (n, N, cache.qk_heads, cache.dk), cache.dtype, dev)
    vp, sv = _drafts("v", v, (n, N, cache.heads, cache.dv), cache.dtype, dev)
    if new_pos is None:
        new_pos = _empty(stream, n, device=cache.device, dtype=torch.int32)
    st = _lib.loglinear_cache_accept(
        cache._ref, _at("slots", slots, torch.int32, (n,), dev), _at("pos", pos, torch.int32, (n,), dev),
        _at("path", path, torch.int32, (n, D), dev), kp, sk, vp, sv,
        _at("log_a", log_a, torch.float32, (n, N, cache.heads), dev),
        _at("new_pos", new_pos, torch.int32, (n,), dev), n, N, D, _raw_stream(stream, dev))
    if st != LL_OK:
        raise LoglinearError(st, "loglinear_cache_accept")
    return new_pos
