"""The oracle of the gated linear recurrence against closed forms and differences (CPU)."""
import numpy as np
import pytest

import oracle


def test_forward_closed_forms():
    T, D = 7, 3
    x = np.arange(T * D, dtype=float).reshape(1, T, D)
    h, state = oracle.glr_forward(x, np.zeros((1, T, D)))
    assert np.array_equal(h, np.cumsum(x, 1)) and np.array_equal(state, h[:, -1])
    # a constant gate: a geometric sum
    la = np.full((1, T, D), np.log(0.5))
    h, _ = oracle.glr_forward(np.ones((1, T, D)), la, "one_minus")
    assert np.allclose(h[0, :, 0], 1 - 0.5 ** np.arange(1, T + 1), rtol=1e-14)
    h, state = oracle.glr_forward(np.zeros((1, T, D)), la, "sqrt", h0=np.full((1, D), 8.0))
    assert np.allclose(state, 8 * 0.5 ** T, rtol=1e-14)


def test_packed_sequences_are_apart():
    rng = np.random.default_rng(0)
    x, la = rng.normal(size=(1, 9, 2)), -rng.random((1, 9, 2))
    cu, h0 = [0, 0, 4, 5, 5, 8], rng.normal(size=(5, 2))
    h, state = oracle.glr_forward(x, la, "sqrt", h0=h0, cu=cu)
    for n in range(5):
        lo, hi = cu[n], cu[n + 1]
        if lo == hi:
            assert np.array_equal(state[n], h0[n])
            continue
        one, last = oracle.glr_forward(x[:, lo:hi], la[:, lo:hi], "sqrt", h0=h0[n:n + 1])
        assert np.array_equal(h[:, lo:hi], one) and np.array_equal(state[n], last[0])
    assert np.isnan(h[0, 8]).all()


@pytest.mark.parametrize("scale", ["none", "one_minus", "sqrt"])
@pytest.mark.parametrize("cu", [None, [0, 3, 3, 4, 9]])
def test_backward_against_differences(scale, cu):
    rng = np.random.default_rng(1)
    B, T, D = (2, 5, 2) if cu is None else (1, 9, 2)
    n = B if cu is None else len(cu) - 1
    x, la = rng.normal(size=(B, T, D)), -0.1 - rng.random((B, T, D))
    h0, dout, ds = rng.normal(size=(n, D)), rng.normal(size=(B, T, D)), rng.normal(size=(n, D))

    def loss(x, la, h0):
        h, state = oracle.glr_forward(x, la, scale, h0=h0, cu=cu)
        return np.nansum(h * dout) + np.sum(state * ds)

    h, _ = oracle.glr_forward(x, la, scale, h0=h0, cu=cu)
    grads = oracle.glr_backward(x, la, h, dout, scale, h0=h0, dstate=ds, cu=cu)
    eps = 1e-6  # central differences: error eps^2 |f'''| / 6 + 1e-16 |f| / eps < 1e-8
    for i, (arr, g) in enumerate(zip((x, la, h0), grads)):
        for at in np.ndindex(arr.shape):
            args = [x, la, h0]
            up, down = arr.copy(), arr.copy()
            up[at] += eps
            down[at] -= eps
            hi = loss(*[up if k == i else v for k, v in enumerate(args)])
            lo = loss(*[down if k == i else v for k, v in enumerate(args)])
            want = 0.0 if np.isnan(g[at]) else g[at]
            assert abs((hi - lo) / (2 * eps) - want) < 1e-7, (i, at)
