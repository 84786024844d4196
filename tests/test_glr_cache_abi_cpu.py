"""Refusals of the recurrence and cache entry points: no GPU, nothing is launched."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from log_linear_attention_fwd_gb300 import _binding
    return _binding


P = ctypes.c_void_p(0x1000)   # never dereferenced: every call here fails validation first
ODD = ctypes.c_void_p(0x1001)


def test_glr_fwd(L):
    f = L.lib().loglinear_glr_fwd
    ok = dict(x=P, xs=None, la=P, ls=None, h0=None, cu=None, N=0, out=P, state=None, B=2, T=10, D=8,
              i=0, g=0, o=0, scale=0, stream=None)

    def call(**kw):
        a = dict(ok, **kw)
        return f(*(a[k] for k in ok))

    assert call(B=-1) == call(T=-1) == call(D=-1) == L.LL_ERR_INVALID
    assert call(i=5) == call(g=-1) == call(o=9) == L.LL_ERR_DTYPE
    assert call(scale=3) == call(scale=-1) == L.LL_ERR_INVALID
    assert call(i=0, g=1) == L.LL_ERR_UNSUPPORTED            # bf16 gates with fp32 inputs
    assert call(x=None) == call(la=None) == call(out=None) == L.LL_ERR_INVALID
    assert call(cu=P, N=3) == L.LL_ERR_INVALID               # packed: B = 1
    assert call(B=1, cu=P, N=-1) == L.LL_ERR_INVALID
    assert call(T=2 ** 30 + 1) == call(B=2 ** 28) == call(D=2 ** 28) == L.LL_ERR_UNSUPPORTED
    assert call(B=2 ** 20, D=2 ** 13) == L.LL_ERR_UNSUPPORTED  # too many clusters
    assert call(x=ODD) == call(la=ODD) == call(out=ODD) == call(h0=ODD) == call(state=ODD) == L.LL_ERR_ALIGN
    assert call(B=1, cu=ODD, N=1) == L.LL_ERR_ALIGN
    assert call(xs=ctypes.byref(L.LLStrides(80, -8, 0))) == L.LL_ERR_INVALID
    assert call(ls=ctypes.byref(L.LLStrides(-80, 8, 0))) == L.LL_ERR_INVALID
    for kw in (dict(B=0), dict(D=0), dict(T=0), dict(B=1, cu=P, N=0)):
        assert call(**kw) == L.LL_OK
        assert call(x=None, la=None, out=None, **kw) == L.LL_OK


@pytest.mark.parametrize("name", ["loglinear_glr_fwd", "loglinear_glr_bwd"])
def test_glr_most_sequences(L, name):
    """The search over the bounds halves the sum of two indices in 32 bits: at most 2^30 sequences.
    D = 0, so that a count that is accepted launches nothing."""
    rest = (P, None) if name == "loglinear_glr_fwd" else (P, P, None, P, P, None)

    def call(N, D):
        return getattr(L.lib(), name)(P, None, P, None, None, P, N, *rest, 1, 10, D, 0, 0, 0, 0, None)

    for N in (2 ** 30 + 1, 2 ** 31 - 2, 2 ** 31 - 1, 2 ** 31, 2 ** 40):
        assert call(N, 0) == call(N, 8) == L.LL_ERR_UNSUPPORTED, N
    assert call(2 ** 30, 0) == L.LL_OK and call(-1, 0) == L.LL_ERR_INVALID


def test_glr_bwd(L):
    f = L.lib().loglinear_glr_bwd
    ok = dict(x=P, xs=None, la=P, ls=None, h0=None, cu=None, N=0, h=P, dout=P, dstate=None, dx=P, dla=P,
              dh0=None, B=2, T=10, D=8, i=0, g=0, o=0, scale=2, stream=None)

    def call(**kw):
        a = dict(ok, **kw)
        return f(*(a[k] for k in ok))

    for name in ("x", "la", "h", "dout", "dx", "dla"):
        assert call(**{name: None}) == L.LL_ERR_INVALID
    for name in ("x", "la", "h", "dout", "dx", "dla", "dstate", "dh0", "h0"):
        assert call(**{name: ODD}) == L.LL_ERR_ALIGN
    assert call(o=7) == L.LL_ERR_DTYPE
    assert call(i=0, g=1) == L.LL_ERR_UNSUPPORTED
    assert call(x=None, scale=0, dout=None) == L.LL_ERR_INVALID   # x is not needed, dout is
    assert call(B=0) == call(T=0) == L.LL_OK


def test_glr_step(L):
    f = L.lib().loglinear_glr_step
    ok = dict(state=P, S=4, slots=P, x=P, la=P, out=P, B=3, D=8, i=0, g=0, o=0, scale=0, stream=None)

    def call(**kw):
        a = dict(ok, **kw)
        return f(*(a[k] for k in ok))

    for name in ("state", "x", "la", "out"):
        assert call(**{name: None}) == L.LL_ERR_INVALID
        assert call(**{name: ODD}) == L.LL_ERR_ALIGN
    assert call(slots=ODD) == L.LL_ERR_ALIGN
    assert call(slots=None, B=5) == L.LL_ERR_SHAPE
    assert call(S=-1) == call(B=-1) == L.LL_ERR_INVALID
    assert call(B=70000, S=70000) == L.LL_ERR_UNSUPPORTED
    assert call(g=1) == L.LL_ERR_UNSUPPORTED
    assert call(B=0, state=None) == call(D=0, x=None) == L.LL_OK


def cache_of(L, **kw):
    a = dict(slots=4, n_pages=8, H=4, Hqk=2, dk=16, dv=8, levels=3, dtype=0, pages=0x1000, page_table=0x1000,
             refcount=0x1000, win_k=0x1000, win_v=0x1000, win_log_a=0x1000, page_log=0x1000, page_from=0x1000,
             scratch=0x1000, error=0x1000)
    a.update(kw)
    return ctypes.byref(L.LLCache(*a.values()))


def test_cache_descriptor(L):
    lib = L.lib()
    call = lambda c, n=2: lib.loglinear_cache_free(c, None, n, None)  # noqa: E731
    assert call(None) == L.LL_ERR_INVALID
    assert call(cache_of(L), -1) == L.LL_ERR_INVALID
    for kw in (dict(slots=0), dict(n_pages=0), dict(H=0), dict(dk=0), dict(dv=0), dict(levels=0),
               dict(Hqk=-1)):
        assert call(cache_of(L, **kw)) == L.LL_ERR_INVALID, kw
    assert call(cache_of(L, Hqk=3)) == call(cache_of(L, Hqk=0)) == L.LL_ERR_SHAPE
    assert call(cache_of(L, dtype=2)) == L.LL_ERR_DTYPE
    for kw in (dict(dk=129), dict(dv=132), dict(dv=6), dict(levels=25), dict(n_pages=2 ** 30 + 1),
               dict(slots=2 ** 30)):
        assert call(cache_of(L, **kw)) == L.LL_ERR_UNSUPPORTED, kw
    assert call(cache_of(L), 2 ** 30) == L.LL_ERR_UNSUPPORTED
    names = ("pages", "page_table", "refcount", "win_k", "win_v", "win_log_a", "page_log", "page_from",
             "scratch", "error")
    for name in names:
        assert call(cache_of(L, **{name: 0})) == L.LL_ERR_INVALID, name
        assert call(cache_of(L, **{name: 0x1002})) == L.LL_ERR_ALIGN, name
    for name in ("pages", "win_k", "win_v"):
        assert call(cache_of(L, **{name: 0x1008})) == L.LL_ERR_ALIGN, name
    assert call(cache_of(L)) == L.LL_ERR_INVALID               # slots NULL
    assert call(cache_of(L), 0) == L.LL_OK
    size = ctypes.c_size_t(0)
    assert lib.loglinear_cache_scratch_size(4, 8, ctypes.byref(size)) == L.LL_OK and size.value >= 4 * (4 + 3 * 8)
    assert lib.loglinear_cache_scratch_size(0, 8, ctypes.byref(size)) == L.LL_ERR_INVALID
    assert lib.loglinear_cache_scratch_size(4, 8, None) == L.LL_ERR_INVALID


def test_cache_calls(L):
    lib, c = L.lib(), cache_of(L)

    def step(c=c, **kw):
        a = dict(slots=P, pos=P, q=P, k=P, v=P, la=None, lam=P, out=P, n=2, L=10, o=0, stream=None)
        a.update(kw)
        return lib.loglinear_cache_step(c, *a.values())

    for name in ("slots", "pos", "q", "k", "v", "lam", "out"):
        assert step(**{name: None}) == L.LL_ERR_INVALID
        assert step(**{name: ODD}) == L.LL_ERR_ALIGN
    assert step(L=9) == L.LL_ERR_SHAPE and step(L=65) == L.LL_ERR_UNSUPPORTED
    assert step(o=3) == L.LL_ERR_DTYPE and step(la=ODD) == L.LL_ERR_ALIGN
    assert step(n=0, q=None) == L.LL_OK and step(n=0, c=None) == L.LL_ERR_INVALID
    assert lib.loglinear_cache_reserve(c, P, None, 2, None) == L.LL_ERR_INVALID
    assert lib.loglinear_cache_reserve(c, ODD, P, 2, None) == L.LL_ERR_ALIGN
    assert lib.loglinear_cache_reserve(c, None, None, 0, None) == L.LL_OK

    def load(**kw):
        a = dict(slots=P, n=2, T=100, state=P, L=8, k=P, ks=None, v=P, vs=None, la=None, las=None, Tk=36,
                 stream=None)
        a.update(kw)
        return lib.loglinear_cache_load(c, *a.values())

    assert load(T=-1) == load(L=0) == load(Tk=-1) == L.LL_ERR_INVALID
    assert load(T=512, L=20) == L.LL_ERR_UNSUPPORTED            # 64 * 2^3 positions do not fit
    assert load(L=7) == L.LL_ERR_SHAPE and load(Tk=35) == L.LL_ERR_SHAPE
    assert load(L=65) == L.LL_ERR_UNSUPPORTED
    for name in ("slots", "state", "k", "v"):
        assert load(**{name: None}) == L.LL_ERR_INVALID
        assert load(**{name: ODD}) == L.LL_ERR_ALIGN
    assert load(state=ctypes.c_void_p(0x1008)) == L.LL_ERR_ALIGN
    assert load(ks=ctypes.byref(L.LLStrides(-1, 1, 1))) == L.LL_ERR_INVALID
    assert load(n=0) == L.LL_OK

    def store(**kw):
        a = dict(slots=P, pos=P, state=P, n=2, L=10, stream=None)
        a.update(kw)
        return lib.loglinear_cache_store(c, *a.values())

    assert store(L=9) == L.LL_ERR_SHAPE and store(L=65) == L.LL_ERR_UNSUPPORTED
    assert store(state=None) == store(pos=None) == L.LL_ERR_INVALID
    assert store(state=ctypes.c_void_p(0x1004)) == L.LL_ERR_ALIGN
    assert lib.loglinear_cache_fork(c, P, None, P, 2, None) == L.LL_ERR_INVALID
    assert lib.loglinear_cache_fork(c, P, P, ODD, 2, None) == L.LL_ERR_ALIGN
    assert lib.loglinear_cache_compact(c, None, None) == L.LL_ERR_INVALID
    assert lib.loglinear_cache_compact(c, ODD, None) == L.LL_ERR_ALIGN
    assert lib.loglinear_cache_compact(None, P, None) == L.LL_ERR_INVALID


def test_binding_refuses_host_tensors(L):
    x = torch.zeros(1, 4, 2)
    with pytest.raises(ValueError):
        L.loglinear_glr_fwd(x, x)
    with pytest.raises(ValueError):
        L.loglinear_glr_step(x[0], x[0], x[0])
    with pytest.raises(ValueError):
        L.LogLinearCache.empty(1, 1, 1, 4, 4, 1, device="cpu")
