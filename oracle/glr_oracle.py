"""fp64 oracle of the gated linear recurrence (test infrastructure only): the definition,
token by token, and its gradients by the chain rule.  No code is shared with the GPU path."""
from __future__ import annotations

import numpy as np


def _f64(x):
    if hasattr(x, "detach"):
        x = x.detach().double().cpu().numpy()
    return np.asarray(x, dtype=np.float64)


def glr_scale(log_a, scale):
    """b(log a) and db / d log a (0 where the square root's derivative is infinite)."""
    la = _f64(log_a)
    if scale == "none":
        return np.ones_like(la), np.zeros_like(la)
    if scale == "one_minus":
        return -np.expm1(la), -np.exp(la)
    b = np.sqrt(np.maximum(-np.expm1(2 * la), 0.0))
    with np.errstate(divide="ignore", invalid="ignore"):
        db = np.where(b > 0, -np.exp(2 * la) / np.where(b > 0, b, 1.0), 0.0)
    return b, db


def _spans(B, T, cu):
    """(batch, first, end, sequence) of every sequence."""
    if cu is None:
        return [(b, 0, T, b) for b in range(B)]
    cu = [int(c) for c in cu]
    return [(0, cu[n], cu[n + 1], n) for n in range(len(cu) - 1)]


def glr_forward(x, log_a, scale="none", h0=None, cu=None):
    """h [B,T,D] (nan where no sequence is) and the last states [N,D]."""
    x, la = _f64(x), _f64(log_a)
    B, T, D = x.shape
    a, (b, _) = np.exp(la), glr_scale(la, scale)
    spans = _spans(B, T, cu)
    state = np.zeros((len(spans), D)) if h0 is None else _f64(h0).copy()
    h = np.full((B, T, D), np.nan)
    for i, lo, hi, n in spans:
        for t in range(lo, hi):
            u = b[i, t] * x[i, t]
            if t > lo or h0 is not None:  # the first token of a sequence without a first state
                u = a[i, t] * state[n] + u
            h[i, t] = state[n] = u
    return h, state


def glr_backward(x, log_a, h, dout, scale="none", h0=None, dstate=None, cu=None):
    """dx, dlog_a [B,T,D] (nan where no sequence is) and dh0 [N,D] from the given h."""
    la, h, dout = _f64(log_a), _f64(h), _f64(dout)
    x = np.zeros_like(la) if x is None else _f64(x)
    B, T, D = la.shape
    a, (b, db) = np.exp(la), glr_scale(la, scale)
    spans = _spans(B, T, cu)
    carry = np.zeros((len(spans), D)) if dstate is None else _f64(dstate).copy()
    first = np.zeros((len(spans), D)) if h0 is None else _f64(h0)
    dx, dla = np.full((B, T, D), np.nan), np.full((B, T, D), np.nan)
    for i, lo, hi, n in spans:
        for t in range(hi - 1, lo - 1, -1):
            g = dout[i, t] + carry[n]
            before = h[i, t - 1] if t > lo else first[n]
            carry[n] = a[i, t] * g
            dx[i, t] = b[i, t] * g
            dla[i, t] = carry[n] * before + db[i, t] * x[i, t] * g
    return dx, dla, carry
