"""The oracle of speculative decoding against things known without it: chains against the
forward's definition, and the law of the verified tokens against the target's distribution."""
import itertools

import numpy as np
import pytest

import oracle
import workloads as W


@pytest.mark.parametrize("T", [0, 1, 63, 64, 70])
def test_a_chain_is_the_forward(T):
    N, H = 9, 2
    cfg = W.FwdConfig("c", 1, H, T + N, 8, 4, 16, 10, "f32", True, "softplus", seed=T, Hqk=1)
    x = W.make_fwd_inputs(cfg)
    y = dict(x, q=x["q"].repeat_interleave(H, 2), k=x["k"].repeat_interleave(H, 2))
    want = oracle.forward_direct(y["q"], y["k"], y["v"], y["log_a"], y["lam"])[0, T:]
    ctx = {n: x[n][0, :T] for n in ("k", "v", "log_a")}
    tree = {n: x[n][0, T:] for n in ("q", "k", "v", "log_a", "lam")}
    got = oracle.tree_attention(ctx, tree, [-1] + list(range(N - 1)))
    np.testing.assert_allclose(got, want, rtol=1e-12, atol=1e-14)


def test_branches_see_their_own_path_only():
    cfg = W.FwdConfig("c", 1, 1, 12, 8, 4, 16, 10, "f32", True, "softplus", seed=3)
    x = W.make_fwd_inputs(cfg)
    ctx = {n: x[n][0, :5] for n in ("k", "v", "log_a")}
    tree = {n: x[n][0, 5:] for n in ("q", "k", "v", "log_a", "lam")}
    parents = [-1, 0, 0, 1, 2, -2, 3]
    got = oracle.tree_attention(ctx, tree, parents)
    assert np.isnan(got[5]).all()
    for i, path in enumerate(oracle.tree_paths(parents)):
        if path is None:
            continue
        line = {n: np.concatenate([np.asarray(ctx[n]), np.asarray(tree[n])[path]])[None] for n in ("k", "v", "log_a")}
        q = np.zeros_like(line["k"])
        q[0, -1] = tree["q"][i]
        lam = np.zeros((1, 5 + len(path), 1, 10))
        lam[0, -1] = tree["lam"][i]
        want = oracle.forward_direct(q, line["k"], line["v"], line["log_a"], lam)[0, -1]
        np.testing.assert_allclose(got[i], want, rtol=1e-12)


@pytest.mark.parametrize("drawn", [True, False])
def test_the_first_new_token_follows_the_target(drawn):
    """Root with two children over a vocabulary of three: the law of the token behind the root,
    summed over the drafts' tokens and integrated over the random numbers on a grid of midpoints,
    is the target's row.  Each number's grid has g points, so every test's probability is off
    by at most 1 / (2 g), three numbers by 1.5 / g together."""
    p, q, g = np.array([0.5, 0.3, 0.2]), np.array([0.2, 0.2, 0.6]), 12
    rows = np.stack([p, [1, 0, 0], [1, 0, 0]])
    grid = (np.arange(g) + 0.5) / g
    law = np.zeros(3)
    pairs = list(itertools.product(range(3), repeat=2)) if drawn else [(2, 0)]
    for x in pairs:
        weight = q[x[0]] * q[x[1]] if drawn else 1.0
        for u in itertools.product(grid, repeat=3):
            path, token = oracle.tree_verify([-1, 0, 0], [0, *x], rows, list(u),
                                             np.stack([q, q, q]) if drawn else None)
            law[x[path[1] - 1] if len(path) > 1 else token] += weight / g ** 3
    np.testing.assert_allclose(law, p, atol=1.5 / g)
    assert abs(law.sum() - 1) < 1e-12


def test_the_walk():
    rows = np.array([[0.0, 1.0, 0.0], [0.0, 0.0, 1.0], [1.0, 0.0, 0.0], [0.2, 0.3, 0.5]])
    path, token = oracle.tree_verify([-1, 0, 1, 2], [0, 1, 2, 0], rows, [0.6, 0.5, 0.5, 0.5])
    assert path == [0, 1, 2, 3] and token == 2
    path, token = oracle.tree_verify([-1, 0, 0, 2], [0, 2, 1, 2], rows, [0.6, 0.5, 0.5, 0.5])
    assert path == [0, 2] and token == 0                       # 1 rejected, 2 taken, 3 rejected
    assert oracle.tree_verify([-2, -2], [0, 0], rows[:2], [0.1, 0.1]) == ([], -1)
