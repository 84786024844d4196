"""fp64 oracle of speculative decoding (test infrastructure only): the attention of a tree of
drafted tokens by the definition, path by path, and the verification walk with its redraws
normalised at every step.  No code is shared with the GPU path."""
from __future__ import annotations

import numpy as np

from .loglinear_oracle import level


def _f64(x):
    if hasattr(x, "detach"):
        x = x.detach().double().cpu().numpy()
    return np.asarray(x, dtype=np.float64)


def tree_paths(parents):
    """Each node's path from its root, itself last; None for a node that is left out."""
    paths = []
    for i, p in enumerate(parents):
        paths.append(None if p == -2 else [i] if p == -1 else paths[p] + [i])
    return paths


def tree_attention(ctx, tree, parents):
    """One row.  ctx: k [T, Hqk, dk], v [T, H, dv], log_a [T, H] or None; tree: q, k [N, Hqk, dk],
    v [N, H, dv], log_a [N, H] or None, lam [N, H, L].  Returns out [N, H, dv], NaN where a node is
    left out."""
    k0, v0 = _f64(ctx["k"]), _f64(ctx["v"])
    q, k, v, lam = (_f64(tree[n]) for n in ("q", "k", "v", "lam"))
    T, H = v0.shape[0], v.shape[1]
    a0 = np.zeros((T, H)) if ctx["log_a"] is None else _f64(ctx["log_a"])
    la = np.zeros((len(parents), H)) if tree["log_a"] is None else _f64(tree["log_a"])
    G = H // q.shape[1]
    out = np.full((len(parents), H, v.shape[2]), np.nan)
    for i, path in enumerate(tree_paths(parents)):
        if path is None:
            continue
        t = T + len(path) - 1
        lev = np.array([level(t, s) for s in range(t + 1)])
        keys, vals = np.concatenate([k0, k[path]]), np.concatenate([v0, v[path]])
        logs = np.concatenate([a0, la[path]])
        for h in range(H):
            back = np.concatenate([np.cumsum(logs[::-1, h])[::-1][1:], [0.0]])  # behind s, up to t
            w = lam[i, h, lev] * np.exp(back) * (keys[:, h // G] @ q[i, h // G])
            out[i, h] = w @ vals[:, h]
    return out


def tree_verify(parents, tokens, probs, u, draft=None):
    """One row: (path, token).  The target's distribution at the current node is normalised again
    after every rejection."""
    if parents[0] == -2:
        return [], -1
    P = np.nan_to_num(_f64(probs), nan=0.0).clip(0, 1)
    Q = None if draft is None else np.nan_to_num(_f64(draft), nan=0.0).clip(0, 1)
    u = np.nan_to_num(_f64(u), nan=0.0).clip(0, 1 - 2.0 ** -24)
    path, cur = [0], 0
    while True:
        left, total, nxt = P[cur].copy(), 1.0, None
        for i in range(cur + 1, len(parents)):
            if parents[i] != cur:
                continue
            x = tokens[i]
            if Q is None:
                if u[i] * total < left[x]:
                    nxt = i
                    break
                total = max(total - left[x], 0.0)
                left[x] = 0.0
            else:
                if u[i] * Q[cur, x] * total < left[x]:
                    nxt = i
                    break
                left = np.maximum(left - total * Q[cur], 0.0)
                total = left.sum()
        if nxt is None:
            break
        path.append(nxt)
        cur = nxt
    if left.sum() <= 0:
        left = P[cur]
    if left.sum() <= 0:
        return path, -1
    cum = np.cumsum(left)
    return path, int(np.argmax(cum > u[0] * cum[-1]))
