"""Refusals of the speculative-decoding entry points: no GPU, nothing is launched."""
import ctypes

import pytest
import torch

from tests.test_glr_cache_abi_cpu import ODD, P, cache_of


@pytest.fixture(scope="module")
def L():
    from log_linear_attention_fwd_gb300 import _binding
    return _binding


def test_cache_tree(L):
    def call(c=cache_of(L), **kw):
        a = dict(slots=P, pos=P, parents=P, q=P, qs=None, k=P, ks=None, v=P, vs=None, la=None, lam=P, out=P, n=2, N=5,
                 L=10, o=0, stream=None)
        a.update(kw)
        return L.lib().loglinear_cache_tree(c, *a.values())

    for name in ("slots", "pos", "parents", "q", "k", "v", "lam", "out"):
        assert call(**{name: None}) == L.LL_ERR_INVALID, name
        assert call(**{name: ODD}) == L.LL_ERR_ALIGN, name
    assert call(la=ODD) == L.LL_ERR_ALIGN
    assert call(L=9) == L.LL_ERR_SHAPE and call(L=65) == L.LL_ERR_UNSUPPORTED
    assert call(N=0) == call(N=-1) == call(n=-1) == call(c=None) == L.LL_ERR_INVALID
    assert call(N=65) == L.LL_ERR_UNSUPPORTED and call(n=2 ** 30) == L.LL_ERR_UNSUPPORTED
    assert call(o=2) == L.LL_ERR_DTYPE and call(c=cache_of(L, dtype=3)) == L.LL_ERR_DTYPE
    for name in ("qs", "ks", "vs"):
        for bad in ((-1, 1, 1), (1, -1, 1), (1, 1, -1)):
            assert call(**{name: ctypes.byref(L.LLStrides(*bad))}) == L.LL_ERR_INVALID
    assert call(n=0, q=None) == L.LL_OK


def test_cache_accept(L):
    def call(c=cache_of(L), **kw):
        a = dict(slots=P, pos=P, path=P, k=P, ks=None, v=P, vs=None, la=None, new=ctypes.c_void_p(0x2000), n=2, N=5,
                 D=4, stream=None)
        a.update(kw)
        return L.lib().loglinear_cache_accept(c, *a.values())

    for name in ("slots", "pos", "path", "k", "v", "new"):
        assert call(**{name: None}) == L.LL_ERR_INVALID, name
        assert call(**{name: ODD}) == L.LL_ERR_ALIGN, name
    assert call(la=ODD) == L.LL_ERR_ALIGN
    assert call(new=P) == L.LL_ERR_INVALID                       # pos itself
    assert call(N=0) == call(D=0) == call(n=-1) == call(c=None) == L.LL_ERR_INVALID
    assert call(N=65) == call(D=65) == L.LL_ERR_UNSUPPORTED
    assert call(ks=ctypes.byref(L.LLStrides(1, -1, 1))) == L.LL_ERR_INVALID
    assert call(n=0, k=None) == L.LL_OK


def test_tree_verify(L):
    def call(**kw):
        a = dict(parents=P, tokens=P, probs=P, draft=None, u=P, path=P, count=P, token=P, n=2, N=5, V=100, dtype=0,
                 stream=None)
        a.update(kw)
        return L.lib().loglinear_tree_verify(*a.values())

    for name in ("parents", "tokens", "probs", "u", "path", "count", "token"):
        assert call(**{name: None}) == L.LL_ERR_INVALID, name
        assert call(**{name: ODD}) == L.LL_ERR_ALIGN, name
    assert call(draft=ODD) == call(probs=ctypes.c_void_p(0x1002)) == L.LL_ERR_ALIGN
    assert call(n=-1) == call(N=0) == call(V=0) == L.LL_ERR_INVALID
    assert call(N=65) == call(V=2 ** 30 + 1) == call(n=2 ** 24 + 1) == L.LL_ERR_UNSUPPORTED
    assert call(dtype=2) == L.LL_ERR_DTYPE
    assert call(n=0, probs=None) == L.LL_OK


def test_binding_refuses_host_tensors(L):
    i = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError):
        L.loglinear_tree_verify(i, i, torch.zeros(2, 3, 5), torch.zeros(2, 3))
