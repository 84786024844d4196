"""Speculative decoding on the GPU: a tree's attention over the paged cache, the verification of
its drafts and the appending of the accepted path, against fp64.

Tolerances as for the cache's step (tests/test_cache_gpu.py): fp32 outputs are sums of up to
a few hundred products of fp32 values whose decays are off by a few 2^-24, rel-L2 below 1e-5.  With bf16
caches the tokens are exact inputs, but a token's weight and a page's value enter their products as two tf32
parts, off by 2^-22: with fp32 outputs another 2^-20 of the scale.  bf16 outputs add their half step, 2^-8 of
each value, and the half step of tf32 at which weights and pages are read, 2^-11 of each product: the signs
are random, so the outputs' rms is the root of the products' sum of squares, and the sum of their
magnitudes is at most sqrt(n) of that, n < 1024 products (4 pages of 128 rows and the tokens): 32 rms.
Tokens, paths and tables are equal.
"""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from tests.helpers import TOL_F32, rel_l2, to64
from tests.test_cache_gpu import DT, i32, invariants, poison, same, snapshot

pytestmark = pytest.mark.gpu
TWO_PARTS, ONE_PART = 2.0 ** -20, 2.0 ** -11


@pytest.fixture(scope="module")
def LL():
    import log_linear_attention_fwd_gb300 as m
    return m


def check(got, want, parts=False):
    got, want = got[~np.isnan(want)], want[~np.isnan(want)]
    if got.dtype == torch.float32:
        tol = TOL_F32 + (TWO_PARTS if parts else 0.0)
        assert rel_l2(got, want) <= tol, rel_l2(got, want)
    else:
        rms = float(np.sqrt(np.mean(np.square(want))))
        off = np.abs(to64(got) - want) - (2.0 ** -8 * np.abs(want) + 32 * (TOL_F32 + (ONE_PART if parts else 0.0)) * rms)
        assert off.max() <= 0, off.max()


def parents_of(n, N, kind, seed=0):
    rng = np.random.default_rng(seed)
    rows = []
    for r in range(n):
        live = N if kind == "chain" else max(1, N - r % 3)
        rows.append([-1] + [-2 if i >= live else i - 1 if kind == "chain" else int(rng.integers(0, i)) if kind == "tree"
                            else int(rng.integers(-1, i)) for i in range(1, N)])
    return rows


def contexts(LL, pos, N, H, Hqk, dk, dv, dtype, decay, M=5, seed=0, slots=None, L=None):
    """A cache whose slots hold pos positions each, the contexts behind them and n trees' inputs."""
    n, L = len(pos), L or M + 7
    slots = slots or [(3 * i + 1) % (n + 2) if (n + 2) % 3 else i for i in range(n)]
    ctx, tree = [], []
    cache = poison(LL.LogLinearCache.empty(n + 2, 4 * n + 2, H, dk, dv, M, Hqk=Hqk, dtype=DT[dtype]))
    for i, T in enumerate(pos):
        cfg = W.FwdConfig("c", 1, H, T + N, dk, dv, 16, L, dtype, decay, "softplus", seed=seed + i, Hqk=Hqk)
        x = W.make_fwd_inputs(cfg)
        ctx.append({k: None if x[k] is None else x[k][0, :T] for k in ("k", "v", "log_a")})
        tree.append({k: None if x[k] is None else x[k][0, T:] for k in ("q", "k", "v", "log_a", "lam")})
        if T:
            d = {k: None if v is None else v[:, :T].cuda().contiguous() for k, v in x.items()}
            _, state = LL.loglinear_prefill(d["q"].float(), d["k"].float(), d["v"].float(), d["log_a"], d["lam"], 16, path="simt")
            tail = lambda t: None if t is None else t[:, max(0, T - 64):]  # noqa: E731
            LL.loglinear_cache_load(cache, i32([slots[i]]), T, state, tail(d["k"]), tail(d["v"]), tail(d["log_a"]))
    assert cache.error() == 0
    x = {k: None if tree[0][k] is None else torch.stack([t[k] for t in tree]).cuda().contiguous() for k in tree[0]}
    return cache, slots, ctx, tree, x


def attend(LL, cache, slots, pos, parents, x, **kw):
    return LL.loglinear_cache_tree(cache, i32(slots), i32(pos), i32(parents), x["q"], x["k"], x["v"], x["log_a"], x["lam"], **kw)


@pytest.mark.parametrize("N,kind", [(1, "tree"), (5, "forest"), (17, "tree"), (64, "chain")])
@pytest.mark.parametrize("H,Hqk,dk,dv,dtype,decay", [
    (2, 2, 16, 8, "f32", True), (4, 2, 33, 20, "bf16", True), (2, 1, 128, 128, "bf16", True), (6, 3, 96, 36, "f32", False),
    (2, 1, 128, 64, "bf16", False), (1, 1, 1, 4, "bf16", True), (2, 2, 128, 128, "f32", True), (1, 1, 72, 100, "bf16", True)])
def test_tree_attention(LL, H, Hqk, dk, dv, dtype, decay, N, kind):
    """Positions at, before and behind blocks' ends, trees that run over them."""
    pos = [0, 1, 63, 64, 127, 150, 448, 511]
    parents = parents_of(len(pos), N, kind)
    cache, slots, ctx, tree, x = contexts(LL, pos, N, H, Hqk, dk, dv, dtype, decay)
    before = snapshot(cache)
    want = np.stack([oracle.tree_attention(c, t, p) for c, t, p in zip(ctx, tree, parents)])
    out = torch.full((len(pos), N, H, dv), 7.0).cuda()
    attend(LL, cache, slots, pos, parents, x, out=out)
    out = out.cpu()
    assert torch.all(out[torch.from_numpy(np.isnan(want))] == 7)
    for r in range(len(pos)):
        check(out[r], want[r], dtype == "bf16")
    got = attend(LL, cache, slots, pos, parents, x, out_dtype=torch.bfloat16).cpu()
    for r in range(len(pos)):
        check(got[r], want[r], dtype == "bf16")
    assert cache.error() == 0
    for a, b in zip(before, snapshot(cache)):
        assert torch.equal(a.nan_to_num(5.0), b.nan_to_num(5.0))


@pytest.mark.parametrize("n,H,Hqk,N,dtype", [(40, 12, 4, 9, "bf16"), (3, 64, 64, 33, "f32"), (170, 1, 1, 3, "bf16")])
def test_more_items_than_sms(LL, n, H, Hqk, N, dtype):
    """Many rows on few slots, idle rows among them."""
    some = [0, 70, 130, 260, 300, 500]
    cache, held, ctx, tree, x = contexts(LL, some, N, H, Hqk, 64, 32, dtype, True)
    pick = [i % 7 for i in range(n)]
    x = {k: v[[min(p, 5) for p in pick]].contiguous() for k, v in x.items()}
    slots, pos = [held[p] if p < 6 else -1 for p in pick], [some[p] if p < 6 else 10 ** 6 for p in pick]
    parents = parents_of(6, N, "tree")
    want = [oracle.tree_attention(c, t, p) for c, t, p in zip(ctx, tree, parents)]
    out = torch.full((n, N, H, 32), 7.0).cuda()
    attend(LL, cache, slots, pos, [parents[min(p, 5)] for p in pick], x, out=out)
    out = out.cpu()
    for r, p in enumerate(pick):
        if p == 6:
            assert torch.all(out[r] == 7)
        else:
            check(out[r], want[p], dtype == "bf16")
    assert cache.error() == 0


@pytest.mark.parametrize("N", [5, 33, 64])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_deep_caches(LL, dtype, N):
    """All 24 levels and positions near 2^29, from random states: chains over a block's end, then accepted."""
    H, Hqk, dk, dv, M = 2, 1, 16, 12, 24
    pos = [(1 << 29) + (1 << 20) + 37 - 64 * i for i in range(2)] + [(64 << M) - 1 - N, (1 << 29) - 2]
    n, L, g = len(pos), M + 7, torch.Generator().manual_seed(N)
    rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    cache = poison(LL.LogLinearCache.empty(n, 25 * n, H, dk, dv, M, Hqk=Hqk, dtype=DT[dtype]))
    x = {"q": rand(n, N, Hqk, dk) / 4, "k": rand(n, N, Hqk, dk) / 4, "v": rand(n, N, H, dv)}
    wk, wv = (rand(n, 64, Hqk, dk) / 4).to(DT[dtype]), rand(n, 64, H, dv).to(DT[dtype])
    x = {k: t.to(DT[dtype]).cuda() for k, t in x.items()}
    x["log_a"], x["lam"] = (-0.05 * torch.rand(n, N, H, generator=g)).cuda(), torch.rand(n, N, H, L, generator=g).cuda()
    wa = -0.05 * torch.rand(n, 64, H, generator=g)
    state = torch.zeros(n, H, L, dk, dv)
    for r, t in enumerate(pos):
        for m in range(M):
            if t >> 6 >> m & 1:
                state[r, :, 7 + m] = rand(H, dk, dv)
        if t & 63:
            LL.loglinear_cache_load(cache, i32([r]), t, state[r:r + 1].cuda(), wk[r:r + 1, 64 - t % 64:].cuda().contiguous(),
                                    wv[r:r + 1, 64 - t % 64:].cuda().contiguous(), wa[r:r + 1, 64 - t % 64:].cuda().contiguous())
    chain = [[i - 1 for i in range(N)]] * n
    want = np.zeros((n, N, H, dv))
    for r, t0 in enumerate(pos):
        held, j = t0 % 64, t0 // 64
        keys = torch.cat([wk[r, 64 - held:], x["k"][r].cpu()]).double().numpy()
        vals = torch.cat([wv[r, 64 - held:], x["v"][r].cpu()]).double().numpy()
        logs = torch.cat([wa[r, 64 - held:], x["log_a"][r].cpu()]).double().numpy()
        S, lam, q = to64(state[r]), to64(x["lam"][r].cpu()), to64(x["q"][r].cpu())
        for i in range(N):
            t, last = t0 + i, held + i
            for h in range(H):
                # a prompt's states are as they are at its last position
                acc = 0.0
                back = logs[:, h].copy()
                since = back[held:last + 1].sum()
                to = ((t // 64) & -(t // 64)).bit_length() - 1 if t // 64 > j else 0
                for m in range(M):
                    if j >> m & 1:
                        acc = acc + lam[i, h, 7 + max(m, to)] * np.exp(since) * (q[i, 0] @ S[h, 7 + m])
                for s in range(last + 1):
                    w = lam[i, h, oracle.level(t, 64 * j + s)] * np.exp(back[s + 1:last + 1].sum()) * (keys[s, 0] @ q[i, 0])
                    acc = acc + w * vals[s, h]
                want[r, i, h] = acc
    for odt in (torch.float32, torch.bfloat16):
        got = attend(LL, cache, list(range(n)), pos, chain, x, out_dtype=odt).cpu()
        for r in range(n):
            check(got[r], want[r], dtype == "bf16")
    assert cache.error() == 0
    # the first half accepted, the second half's nodes behind them: as before
    half = (N + 1) // 2
    new = LL.loglinear_cache_accept(cache, i32(list(range(n))), i32(pos), i32([list(range(half)) + [-1]] * n), x["k"], x["v"], x["log_a"])
    assert new.tolist() == [p + half for p in pos] and cache.error() == 0
    rest = {k: t[:, half:].contiguous() for k, t in x.items()}
    got = attend(LL, cache, list(range(n)), new.tolist(), [[i - 1 for i in range(N - half)]] * n, rest, out_dtype=torch.float32).cpu()
    for r in range(n):
        check(got[r], want[r, half:], dtype == "bf16")
    assert cache.error() == 0


def test_pages_past_32_bits(LL):
    """Pages, keys and values whose offsets in elements pass 2^32: low pages taken, high slots."""
    H, Hqk, d, M, slots = 16, 16, 128, 3, 33000
    n_pages = 16600                                            # of 2^18 elements
    cache = LL.LogLinearCache.empty(slots, n_pages, H, d, d, M, Hqk=Hqk)
    low = n_pages - 6
    assert low * H * d * d > 2 ** 32 and (slots - 2) * H * 64 * d > 2 ** 32
    cache.refcount[:low] = 1
    N, pos, s = 9, [120, 186], [slots - 1, slots - 2]
    ctx, tree = [], []
    for i, T in enumerate(pos):
        x = W.make_fwd_inputs(W.FwdConfig("c", 1, H, T + N, d, d, 16, M + 7, "bf16", True, "softplus", seed=i, Hqk=Hqk))
        ctx.append({k: x[k][0, :T] for k in ("k", "v", "log_a")})
        tree.append({k: x[k][0, T:] for k in ("q", "k", "v", "log_a", "lam")})
        c = {k: v[:, :T].cuda().contiguous() for k, v in x.items()}
        _, state = LL.loglinear_prefill(c["q"].float(), c["k"].float(), c["v"].float(), c["log_a"], c["lam"], 16, path="simt")
        LL.loglinear_cache_load(cache, i32([s[i]]), T, state, c["k"][:, -64:], c["v"][:, -64:], c["log_a"][:, -64:])
    x = {k: torch.stack([t[k] for t in tree]).cuda().contiguous() for k in tree[0]}
    chain = [[i - 1 for i in range(N)]] * 2
    want = [oracle.tree_attention(c, t, p) for c, t, p in zip(ctx, tree, chain)]
    got = attend(LL, cache, s, pos, chain, x, out_dtype=torch.float32).cpu()
    for r in range(2):
        check(got[r], want[r], True)
    new = LL.loglinear_cache_accept(cache, i32(s), i32(pos), i32([list(range(8))] * 2), x["k"], x["v"], x["log_a"])
    assert new.tolist() == [128, 194] and cache.error() == 0
    assert min(cache.page_table[s[0]].max().item(), cache.page_table[s[1]].max().item()) >= low
    last = {k: t[:, 8:].contiguous() for k, t in x.items()}
    got = attend(LL, cache, s, new.tolist(), [[-1]] * 2, last, out_dtype=torch.float32).cpu()
    for r in range(2):
        check(got[r], want[r][8:], True)


def test_no_rows(LL):
    cache = LL.LogLinearCache.empty(2, 2, 2, 16, 8, 2)
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt).cuda()  # noqa: E731
    none = i32([])
    k, v, la = z(0, 3, 2, 16), z(0, 3, 2, 8), z(0, 3, 2, dt=torch.float32)
    empty = torch.zeros(0, 3, dtype=torch.int32).cuda()
    assert LL.loglinear_cache_tree(cache, none, none, empty, k, k, v, la, z(0, 3, 2, 9, dt=torch.float32)).shape == (0, 3, 2, 8)
    assert LL.loglinear_cache_accept(cache, none, none, empty, k, v, la).shape == (0,)
    path, count, token = LL.loglinear_tree_verify(empty, empty, z(0, 3, 5), z(0, 3, dt=torch.float32))
    assert path.shape == (0, 3) and count.shape == token.shape == (0,)
    assert cache.error() == 0 and LL.device_error() == 0


def test_a_tree_of_one_is_a_step(LL):
    pos = [5, 63, 127, 200]
    cache, slots, ctx, tree, x = contexts(LL, pos, 1, 2, 1, 128, 64, "bf16", True)
    got = attend(LL, cache, slots, pos, [[-1]] * 4, x, out_dtype=torch.float32)
    LL.loglinear_cache_reserve(cache, i32(slots), i32(pos))
    one = {k: v[:, 0].contiguous() for k, v in x.items()}
    want = LL.loglinear_cache_step(cache, i32(slots), i32(pos), one["q"], one["k"], one["v"], one["log_a"], one["lam"], out_dtype=torch.float32)
    for r in range(4):
        check(got[r, 0].cpu(), to64(want[r]), True)


def test_strided_drafts(LL):
    """q, k and v as slices of one projection, at an odd offset too (no 16-byte alignment)."""
    n, N, H, d = 3, 6, 4, 64
    pos = [40, 64, 300]
    cache, slots, ctx, tree, x = contexts(LL, pos, N, H, H, d, d, "bf16", True)
    parents = parents_of(n, N, "tree")
    zeros = lambda: torch.zeros(n, N, H, d, dtype=torch.bfloat16).cuda()  # noqa: E731  (left-out nodes are not written)
    want = attend(LL, cache, slots, pos, parents, x, out=zeros())
    for extra in (0, 1, 8):
        wide = torch.full((n, N, H, 3 * d + extra), float("nan"), dtype=torch.bfloat16).cuda()
        y = dict(x)
        for i, name in enumerate("qkv"):
            y[name] = wide[..., extra + i * d:extra + (i + 1) * d]
            y[name].copy_(x[name])
        assert torch.equal(attend(LL, cache, slots, pos, parents, y, out=zeros()), want)
        one = snapshot(cache)
        paths = i32([[0, 1, -1], [0, -1, 3], [2, 2, 5]])
        twin, other = LL.LogLinearCache(*one), LL.LogLinearCache(*snapshot(cache))
        a = LL.loglinear_cache_accept(twin, i32(slots), i32(pos), paths, x["k"], x["v"], x["log_a"])
        b = LL.loglinear_cache_accept(other, i32(slots), i32(pos), paths, y["k"], y["v"], y["log_a"])
        assert torch.equal(a, b) and a.tolist() == [42, 65, 303] and same(snapshot(twin), snapshot(other))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_other_branches_do_not_matter(LL, dtype, bad):
    """What stands in other branches, in nodes that are left out and in stale places of the block
    changes nothing, to the bit."""
    pos, N = [70, 130], 9
    parents = [[-1, 0, 0, 1, 2, 2, -2, 4, -2], [-1, 0, 1, 2, 3, -1, 5, -2, 6]]
    cache, slots, ctx, tree, x = contexts(LL, pos, N, 2, 1, 64, 32, dtype, True)
    want = attend(LL, cache, slots, pos, parents, x)
    for r, up in enumerate(parents):
        paths = oracle.tree_paths(up)
        for hit in (2, 5, 6):
            y = {k: v.clone() for k, v in x.items()}
            for name in "qkv":
                y[name][r, hit] = bad
            y["lam"][r, hit] = bad
            got = attend(LL, cache, slots, pos, parents, y)
            for i, path in enumerate(paths):
                if path is not None and hit not in path:
                    assert torch.equal(got[r, i], want[r, i]), (r, hit, i)
            assert torch.equal(got[1 - r][[p is not None for p in oracle.tree_paths(parents[1 - r])]],
                               want[1 - r][[p is not None for p in oracle.tree_paths(parents[1 - r])]])


@pytest.mark.parametrize("where", ["page", "window", "node", "query"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_infinities_come_out_as_in_the_sum(LL, dtype, where):
    """One infinite value: outputs that it reaches are the infinity of the sum itself, the others
    finite."""
    pos, N, H, dk, dv = [130], 6, 1, 32, 16
    cache, slots, ctx, tree, x = contexts(LL, pos, N, H, H, dk, dv, dtype, True)
    for name in ("q", "k"):
        x[name].abs_()
    cache.win_k.abs_()
    x["q"].clamp_(min=0.125)
    x["k"].clamp_(min=0.125)
    parents = [[-1, 0, 1, 1, 2, 0]]
    inf, s = float("inf"), slots[0]
    if where == "page":
        cache.pages[cache.page_table[s, 1], 0, 3, 5] = -inf
        hit = np.zeros((N, dv), bool)
        hit[:, 5] = True
    elif where == "window":
        cache.win_k[s, 0, :2].clamp_(min=0.125)
        cache.win_v[s, 0, 1, 7] = -inf
        hit = np.zeros((N, dv), bool)
        hit[:, 7] = True
    elif where == "node":
        x["v"][0, 2, 0, 9] = -inf
        hit = np.zeros((N, dv), bool)
        hit[[2, 4], 9] = True
    else:
        x["q"][0, 3, 0, :] = 0
        x["q"][0, 3, 0, 1] = inf
        hit = None
    got = attend(LL, cache, slots, pos, parents, x, out_dtype=torch.float32).cpu().numpy()[0, :, 0]
    if hit is not None:
        assert np.all(got[hit] == -inf), got[hit]
        assert np.isfinite(got[~hit]).all()
    else:
        assert np.isfinite(got[[0, 1, 2, 4, 5]]).all() and not np.isfinite(got[3]).any()


def test_resets_in_a_tree(LL):
    """log a of -inf (a = 0) and the lowest value on a path drop all that came before."""
    pos, N = [70], 6
    cache, slots, ctx, tree, x = contexts(LL, pos, N, 2, 2, 16, 8, "f32", True)
    parents = [[-1, 0, 1, 2, 3, 1]]
    x["log_a"][0, 1], x["log_a"][0, 3] = -float("inf"), torch.finfo(torch.float32).min
    tree[0]["log_a"] = x["log_a"][0].cpu().clamp(min=-1e4)
    want = oracle.tree_attention(ctx[0], tree[0], parents[0])
    check(attend(LL, cache, slots, pos, parents, x)[0].cpu(), want)
    paths = i32([[0, 1, 2]])
    new = LL.loglinear_cache_accept(cache, i32(slots), i32(pos), paths, x["k"], x["v"], x["log_a"])
    after = attend(LL, cache, slots, new.tolist(), [[-1] * N], x)
    ctx[0] = {n: torch.cat([ctx[0][n], tree[0][n][:3]]) for n in ctx[0]}
    check(after[0].cpu(), oracle.tree_attention(ctx[0], tree[0], [-1] * N))


def test_rows_that_cannot_be_served(LL):
    pos, N = [70, 130, 64], 4
    cache, slots, ctx, tree, x = contexts(LL, pos, N, 2, 2, 16, 8, "f32", True)
    good = [-1, 0, 1, -2]
    M = cache.levels
    top = 64 * 2 ** M - 1
    want = [oracle.tree_attention(c, t, good) for c, t in zip(ctx, tree)]

    def run(slots, pos, parents, bits):
        out = torch.full((3, N, 2, 8), 7.0).cuda()
        attend(LL, cache, slots, pos, parents, x, out=out)
        assert cache.error() == bits
        return out.cpu()

    for up in ([-1, 1, 0, 0], [-1, 2, 0, 0], [-1, 0, -3, 0], [-1, -2, 1, -1], [0, 0, 0, 0], [-2, 0, 1, 1], [-1, 0, 2 ** 31 - 1, 0], [-1, 0, -2 ** 31, 0]):
        out = run(slots, pos, [good, up, good], LL.CACHE_ERR_TREE)
        assert torch.all(out[1] == 7)
        check(out[0], want[0])
        check(out[2], want[2])
    out = run([slots[0], 5, -7], pos, [good] * 3, LL.CACHE_ERR_SLOT)
    check(out[0], want[0])
    assert torch.all(out[1:] == 7)
    for bad in (-1, top, top - 2, 2 ** 31 - 1):
        out = run(slots, [bad, pos[1], pos[2]], [good] * 3, LL.CACHE_ERR_POSITION if bad != top - 2 else LL.CACHE_ERR_MISSING | LL.CACHE_ERR_POSITION)
        assert torch.all(out[0] == 7)
    assert torch.all(run([-1, -1, -1], [-5, top, 0], [[5] * 4] * 3, 0) == 7)
    out = run(slots, [70, 129, 64], [good] * 3, LL.CACHE_ERR_POSITION)      # before the end of the loaded prompt
    assert torch.all(out[1] == 7)
    keep = cache.page_table[slots[1], 1].item()
    for e in (-1, 10 ** 6, -7):
        cache.page_table[slots[1], 1] = e
        out = run(slots, pos, [good] * 3, LL.CACHE_ERR_MISSING)
        assert torch.all(out[1] == 7)
    cache.page_table[slots[1], 1] = keep
    # a tree may end at the last position there is
    check(run(slots, pos, [good] * 3, 0)[1], want[1])


# ---------------------------------------------------------------- accept

def steps(LL, cache, slots, pos, paths, x):
    """The path by single steps."""
    pos = list(pos)
    for r, path in enumerate(paths):
        for node in path:
            if node < 0 or slots[r] < 0:
                break
            s, p = i32([slots[r]]), i32([pos[r]])
            LL.loglinear_cache_reserve(cache, s, p)
            a = {k: None if v is None else v[r:r + 1, node].contiguous() for k, v in x.items()}
            LL.loglinear_cache_step(cache, s, p, a["q"], a["k"], a["v"], a["log_a"], a["lam"])
            pos[r] += 1
    return pos


@pytest.mark.parametrize("H,Hqk,dk,dv,dtype,decay", [
    (2, 2, 16, 8, "f32", True), (4, 2, 33, 20, "bf16", True), (2, 1, 128, 128, "bf16", True), (6, 3, 96, 36, "f32", False),
    (2, 1, 128, 64, "bf16", False), (1, 1, 1, 4, "bf16", True), (6, 2, 128, 128, "f32", True), (1, 1, 72, 104, "bf16", True)])
def test_accept_is_the_steps(LL, H, Hqk, dk, dv, dtype, decay):
    """The path's nodes as single steps would have left them: tokens to the bit, folds as sums, and the same
    outputs from there on."""
    pos = [0, 60, 63, 64, 126, 127, 200, 255, 447, 510]
    N, D = 12, 7
    paths = [[0, 3, 4, -1, 9, 9, 9], [2, 5, 7, 11, -1, -1, -1], [1, -1, -1, -1, -1, -1, -1], [-1] * 7, [0, 1, 2, 3, 4, 5, 6], [4, 4, 4, -1, -1, -1, -1],
             [11, 10, 9, 8, 7, 6, 5], [0, 2, -1, -1, -1, -1, -1], [3, 6, -1, -1, -1, -1, -1], [1, 2, -1, -1, -1, -1, -1]]
    cache, slots, ctx, tree, x = contexts(LL, pos, N, H, Hqk, dk, dv, dtype, decay)
    slots[6] = -1
    twin = LL.LogLinearCache(*snapshot(cache))
    new = LL.loglinear_cache_accept(cache, i32(slots), i32(pos), i32(paths), x["k"], x["v"], x["log_a"], new_pos=i32([-5] * 10))
    got = new.tolist()
    end = steps(LL, twin, slots, pos, paths, x)
    assert got == [(-5 if slots[r] < 0 else p) for r, p in enumerate(end)]
    assert cache.error() == 0 and twin.error() == 0
    LL.loglinear_cache_reserve(cache, i32(slots), i32(end))
    LL.loglinear_cache_reserve(twin, i32(slots), i32(end))
    live = {s: p for s, p in zip(slots, end) if s >= 0}
    assert torch.equal(cache.page_table >= 0, twin.page_table >= 0)
    for s, p in live.items():
        r, j = p % 64, p // 64
        assert same([t[s, :, :r] for t in (cache.win_k, cache.win_v, cache.win_log_a)],
                    [t[s, :, :r] for t in (twin.win_k, twin.win_v, twin.win_log_a)])
        for m in range(cache.levels):
            if j >> m & 1:
                a, b = (c.pages[int(c.page_table[s, m])] for c in (cache, twin))
                assert rel_l2(a, to64(b)) <= TOL_F32
                u, w = (c.page_log[s, j & 1, m] for c in (cache, twin))
                np.testing.assert_allclose(to64(u), to64(w), rtol=1e-6, atol=1e-7)
        assert cache.page_from[s, j & 1] == twin.page_from[s, j & 1]
    a, b = (attend(LL, c, slots, end, parents_of(10, N, "chain"), x, out=torch.zeros(10, N, H, dv).cuda()) for c in (cache, twin))
    assert rel_l2(a, to64(b)) <= TOL_F32
    # and against the definition
    for row in (4, 8):
        path = [i for i in paths[row] if i >= 0]
        after = {n: None if ctx[row][n] is None else torch.cat([ctx[row][n], tree[row][n][path]]) for n in ctx[row]}
        check(a[row].cpu(), oracle.tree_attention(after, tree[row], parents_of(1, N, "chain")[0]), dtype == "bf16")


def test_the_longest_path(LL):
    """64 nodes from every place in a block."""
    pos = [0, 1, 37, 62, 63, 64]
    cache, slots, ctx, tree, x = contexts(LL, pos, 64, 1, 1, 16, 8, "bf16", True)
    path = [list(range(64))] * 6
    twin = LL.LogLinearCache(*snapshot(cache))
    new = LL.loglinear_cache_accept(cache, i32(slots), i32(pos), i32(path), x["k"], x["v"], x["log_a"])
    assert new.tolist() == [p + 64 for p in pos] and cache.error() == 0
    steps(LL, twin, slots, pos, path, x)
    up = [[-1] * 64] * 6
    a, b = (attend(LL, c, slots, new.tolist(), up, x, out_dtype=torch.float32) for c in (cache, twin))
    assert rel_l2(a, to64(b)) <= TOL_F32


def test_accept_may_be_repeated_with_other_drafts(LL):
    """Up to a block's end included; the fold is made again from what then stands there."""
    pos, N = [58, 120], 8
    cache, slots, ctx, tree, x = contexts(LL, pos, N, 2, 1, 32, 16, "bf16", True)
    twin = LL.LogLinearCache(*snapshot(cache))
    LL.loglinear_cache_accept(cache, i32(slots), i32(pos), i32([[7, 6, 5, 4, 3, 2], [1, 1, 1, 1, 1, 1]]), x["k"], x["v"], x["log_a"])
    for c in (cache, twin):
        LL.loglinear_cache_accept(c, i32(slots), i32(pos), i32([[0, 1, 2, 3, 4, 5], [0, 1, 2, 3, 4, 5]]), x["k"], x["v"], x["log_a"])
    up = [[-1] * N] * 2
    a, b = (attend(LL, c, slots, [64, 126], up, x) for c in (cache, twin))
    assert torch.equal(a, b) and cache.error() == 0


def test_accept_rows_that_cannot_be_served(LL):
    pos, N = [70, 126, 63], 4
    cache, slots, ctx, tree, x = contexts(LL, pos, N, 2, 2, 16, 8, "f32", True)
    M = cache.levels
    top = 64 * 2 ** M - 1

    def run(bits, left, slots=slots, pos=pos, paths=[[0, 1, 2], [0, 1, 2], [0, 1, 2]]):
        c = LL.LogLinearCache(*snapshot(cache))
        new = LL.loglinear_cache_accept(c, i32(slots), i32(pos), i32(paths), x["k"], x["v"], x["log_a"], new_pos=i32([-9] * 3))
        assert c.error() == bits
        assert new.tolist() == [-9 if r in left else pos[r] + 3 for r in range(3)]
        for r in left:
            if 0 <= slots[r] < c.slots and slots.index(slots[r]) == r:
                s = slots[r]
                assert same([t[s].nan_to_num(5.0) for t in (c.win_k, c.win_v, c.win_log_a)],
                            [t[s].nan_to_num(5.0) for t in (cache.win_k, cache.win_v, cache.win_log_a)])
        return c

    run(0, [])
    for bad in (4, -2, 2 ** 31 - 1, -2 ** 31):
        run(LL.CACHE_ERR_TREE, [1], paths=[[0, 1, 2], [0, 1, bad], [0, 1, 2]])
        run(LL.CACHE_ERR_TREE, [0], paths=[[bad, 1, 2], [0, 1, 1], [0, 1, 2]])
    run(LL.CACHE_ERR_SLOT, [1], slots=[slots[0], slots[0], slots[2]])
    run(LL.CACHE_ERR_SLOT, [0, 2], slots=[99, slots[1], -4])
    run(0, [1], slots=[slots[0], -1, slots[2]])
    for bad in (-1, top, top - 2, 2 ** 31 - 1):
        run(LL.CACHE_ERR_POSITION, [0], pos=[bad, pos[1], pos[2]])
    run(LL.CACHE_ERR_POSITION, [0], pos=[69, pos[1], pos[2]])               # before the end of the loaded prompt
    cache.page_table[slots[1], 0] = -1                                       # a page that the fold needs
    run(LL.CACHE_ERR_MISSING, [1])
    cache.page_table[slots[1], 0] = 10 ** 6
    run(LL.CACHE_ERR_MISSING, [1])
    cache.page_table[slots[1], 0] = -1
    cache.refcount.fill_(1)                                                   # no page is free
    run(LL.CACHE_ERR_PAGES | LL.CACHE_ERR_MISSING, [1, 2])


def test_accept_on_a_fork_leaves_its_source(LL):
    """Shared pages stay; a page left over where the fold goes, and shared, is replaced."""
    pos, N = [125], 6
    cache, slots, ctx, tree, x = contexts(LL, pos, N, 2, 2, 16, 8, "f32", True)
    a, b = slots[0], (slots[0] + 1) % cache.slots
    LL.loglinear_cache_fork(cache, i32([a]), i32([b]), i32(pos))
    want = oracle.tree_attention(ctx[0], tree[0], [-1] * N)
    LL.loglinear_cache_accept(cache, i32([b]), i32(pos), i32([[0, 1, 2, 3, 4]]), x["k"], x["v"], x["log_a"])
    check(attend(LL, cache, [a], pos, [[-1] * N], x)[0].cpu(), want)
    after = {n: torch.cat([ctx[0][n], tree[0][n][:5]]) for n in ctx[0]}
    check(attend(LL, cache, [b], [130], [[-1] * N], x)[0].cpu(), oracle.tree_attention(after, tree[0], [-1] * N))
    assert cache.error() == 0


@pytest.mark.parametrize("n", [1024, 1100])
def test_accept_more_rows_than_a_plan_has_threads(LL, n):
    H, dk, dv, M = 1, 4, 4, 2
    cache = LL.LogLinearCache.empty(n + 5, n, H, dk, dv, M, dtype=torch.float32)
    g = torch.Generator().manual_seed(0)
    k, v = torch.randn(n, 3, H, dk, generator=g).cuda(), torch.randn(n, 3, H, dv, generator=g).cuda()
    slots = torch.randperm(n, generator=g).to(torch.int32)
    slots[700] = slots[3]
    slots[800] = -1
    path = [[0, 1, -1] if r % 3 else [2, 9, 0] if r == 900 else [1, 2, 0] for r in range(n)]
    pos = [62] * n
    new = LL.loglinear_cache_accept(cache, slots.cuda(), i32(pos), i32(path), k, v, None, new_pos=i32([0] * n)).tolist()
    assert cache.error() == LL.CACHE_ERR_SLOT | LL.CACHE_ERR_TREE
    assert [r for r in range(n) if new[r] == 0] == [700, 800, 900]
    assert all(new[r] == 62 + (2 if r % 3 else 3) for r in range(n) if r not in (700, 800, 900))
    table = cache.page_table[:, 0].cpu()
    taken = [int(table[slots[r]]) for r in range(n) if r not in (700, 800, 900)]
    assert taken == list(range(n - 3))                                        # lowest first, in the order of the rows


# ---------------------------------------------------------------- verify

def drafts(n, N, V, dtype, drawn, seed=0, offset=0):
    g = torch.Generator().manual_seed(seed)
    a = 2 * torch.randn(n, N, V, generator=g)
    draft = torch.softmax(a, -1).to(DT[dtype])
    probs = torch.softmax(a + 0.7 * torch.randn(n, N, V, generator=g), -1).to(DT[dtype])
    parents = parents_of(n, N, "tree", seed)
    tokens = [[0] * N for _ in range(n)]
    for r in range(n):
        for i in range(1, N):
            row = draft[r, max(parents[r][i], 0)].double()
            tokens[r][i] = int(torch.multinomial(row, 1, generator=g)) if drawn else int(row.topk(min(V, 1 + i % 3)).indices[-1])
    return parents, tokens, probs, torch.rand(n, N, generator=g), draft if drawn else None


def at_offset(t, offset):
    if t is None:
        return None
    room = torch.empty(t.numel() + offset, dtype=t.dtype).cuda()
    return room[offset:].view(t.shape).copy_(t)


def verify(LL, parents, tokens, probs, u, draft, offsets=(0, 0), **kw):
    return LL.loglinear_tree_verify(i32(parents), i32(tokens), at_offset(probs, offsets[0]), u.cuda().float(),
                                    draft=at_offset(draft, offsets[1]), **kw)


def check_verify(got, parents, tokens, probs, u, draft):
    path, count, token = (t.tolist() for t in got)
    for r in range(len(parents)):
        want, nxt = oracle.tree_verify(parents[r], tokens[r], probs[r], u[r], None if draft is None else draft[r])
        assert path[r] == want + [-1] * (len(parents[r]) - len(want)), r
        assert count[r] == len(want) and token[r] == nxt, (r, token[r], nxt)


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,N,V", [(5, 1, 1), (4, 2, 2), (6, 7, 5), (9, 64, 37), (12, 12, 1000), (3, 5, 50021), (2, 4, 131073), (200, 3, 257)])
def test_verify(LL, n, N, V, dtype, drawn):
    x = drafts(n, N, V, dtype, drawn, seed=n + V)
    check_verify(verify(LL, *x), *x)
    assert LL.device_error() == 0


@pytest.mark.parametrize("offsets", [(1, 1), (1, 0), (3, 5), (0, 2)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_verify_at_any_alignment(LL, dtype, offsets):
    for V in (999, 4096):
        x = drafts(4, 6, V, dtype, True, seed=V)
        check_verify(verify(LL, *x, offsets=offsets), *x)


@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_verify_long_runs(LL, dtype, offset):
    """Warps' runs of more than 1024 values, at their borders: every row's next token where u_0 puts it."""
    n, V = 40, 70001
    g = torch.Generator().manual_seed(offset)
    for drawn in (False, True):
        probs = torch.softmax(torch.randn(n, 2, V, generator=g), -1).to(DT[dtype])
        draft = torch.softmax(torch.randn(n, 2, V, generator=g), -1).to(DT[dtype]) if drawn else None
        tokens = [[0, int(torch.randint(V, (1,), generator=g))] for _ in range(n)]
        u = torch.stack([torch.linspace(0, 1 - 2.0 ** -24, n), torch.full((n,), 1 - 2.0 ** -24)], 1)
        x = ([[-1, 0]] * n, tokens, probs, u, draft)
        check_verify(verify(LL, *x, offsets=(offset, offset)), *x)


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,V", [(3, 9001), (700, 300)])
def test_verify_many_siblings(LL, n, V, dtype, drawn):
    """All 63 drafts behind one node, tokens among them twice, hard to accept: by clusters and by single CTAs."""
    N = 64
    _, _, probs, u, draft = drafts(n, N, V, dtype, drawn, seed=V)
    g = torch.Generator().manual_seed(n)
    tokens = [[0] + torch.multinomial(draft[r, 0].double() if drawn else torch.ones(100, dtype=torch.float64), N - 1,
                                      replacement=True, generator=g).tolist() for r in range(n)]
    if not drawn:
        assert max(len(t) - len(set(t)) for t in tokens) > 5
    u = 1 - u ** 4 / 16
    u[:, 0] = torch.rand(n, generator=g)
    parents = [[-1] + [0] * (N - 1)] * n
    got = LL.loglinear_tree_verify(i32(parents), i32(tokens), probs.cuda(), u.cuda(), draft=None if draft is None else draft.cuda())
    check_verify(got, parents, tokens, probs, u, draft)
    assert LL.device_error() == 0


def test_two_streams_at_once(LL):
    """Trees of one cache and verifications, at once on two streams, eager and as graphs: as by themselves."""
    pos, N = [70, 126, 300], 12
    cache, slots, ctx, tree, x = contexts(LL, pos, N, 4, 2, 64, 32, "bf16", True)
    plans = [parents_of(3, N, "tree", 1), parents_of(3, N, "forest", 2)]
    dr = [drafts(6, 9, 5003, "f32", True, seed=i) for i in range(2)]
    dr = [(i32(p), i32(t), q.cuda(), u.cuda(), d.cuda()) for p, t, q, u, d in dr]
    outs = [torch.zeros(3, N, 4, 32).cuda() for _ in range(2)]
    res = [None, None]

    dev = [(i32(slots), i32(pos), i32(p)) for p in plans]

    def call(i):
        LL.loglinear_cache_tree(cache, *dev[i], x["q"], x["k"], x["v"], x["log_a"], x["lam"], out=outs[i])
        res[i] = LL.loglinear_tree_verify(*dr[i][:4], draft=dr[i][4])

    want = []
    for i in range(2):
        call(i)
        torch.cuda.synchronize()
        want.append((outs[i].clone(), *[t.clone() for t in res[i]]))
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i)
        graphs.append((g, res[i]))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for graph in (False, True):
        for i in range(2):
            outs[i].zero_()
        torch.cuda.synchronize()
        for _ in range(20):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    graphs[i][0].replay() if graph else call(i)
        torch.cuda.synchronize()
        for i in range(2):
            got = (outs[i], *(graphs[i][1] if graph else res[i]))
            assert all(torch.equal(p, q) for p, q in zip(got, want[i]))
    assert cache.error() == 0 and LL.device_error() == 0


def test_verify_repeats_and_does_not_depend_on_the_batch(LL):
    x = drafts(7, 9, 20011, "f32", True, seed=5)
    whole = [t.clone() for t in verify(LL, *x)]
    for r in range(7):
        one = verify(LL, x[0][r:r + 1], x[1][r:r + 1], x[2][r:r + 1], x[3][r:r + 1], x[4][r:r + 1])
        assert all(torch.equal(a[r:r + 1], b) for a, b in zip(whole, one))


def test_verify_borders(LL):
    """Equal distributions accept all; numbers at and outside the borders; rows of zeros, ones, NaN and
    negative values; repeated siblings; tokens of no mass."""
    V, N = 40, 5
    parents = [[-1, 0, 0, 1, 3]]
    g = torch.Generator().manual_seed(1)
    p = torch.softmax(torch.randn(1, N, V, generator=g), -1)
    for u in (0.0, 0.5, 1 - 2 ** -24, 1.0, 7.0, -1.0, float("nan"), float("inf")):
        us = torch.full((1, N), u)
        x = (parents, [[0, 3, 3, 5, 7]], p, us, p.clone())
        got = verify(LL, *x)
        assert got[0].tolist() == [[0, 1, 3, 4, -1]] and got[1].tolist() == [3 + 1]
        check_verify(got, *x)
        x = (parents, [[0, 3, 3, 5, 7]], p, us, None)
        check_verify(verify(LL, *x), *x)
    zero, one_hot = torch.zeros(1, N, V), torch.nn.functional.one_hot(torch.full((1, N), 9), V).float()
    odd = p.clone()
    odd[..., 4], odd[..., 6], odd[..., 8] = float("nan"), -0.5, 1.5
    for probs in (zero, one_hot, odd):
        for draft in (None, p, one_hot, zero):
            for u in (0.0, 0.3, 0.999):
                x = (parents, [[0, 9, 8, 9, 4]], probs, torch.full((1, N), u), draft)
                check_verify(verify(LL, *x), *x)
    assert verify(LL, parents, [[0, 9, 8, 9, 4]], zero, torch.zeros(1, N), None)[2].tolist() == [-1]
    assert LL.device_error() == 0


@pytest.mark.parametrize("V", [30, 9001])
def test_verify_rows_that_are_no_trees(LL, V):
    n, N = 4, 4
    x = drafts(n, N, V, "f32", True, seed=2)
    good = x[0][0]
    for up, tok in (([-1, 1, 0, 0], None), ([-1, 0, -3, 0], None), ([0, 0, 0, 0], None), ([-1, -2, 1, 0], None),
                    ([-2, 0, 0, 0], None), ([-1, 2 ** 31 - 1, 0, 0], None), (good, V), (good, -1), (good, 2 ** 31 - 1)):
        parents, tokens = [list(r) for r in x[0]], [list(r) for r in x[1]]
        parents[1] = up
        if tok is not None:
            tokens[1][1] = tok
        path, count, token = verify(LL, parents, tokens, *x[2:])
        assert LL.device_error() == 32
        assert path[1].tolist() == [-1] * N and count[1] == 0 and token[1] == -1
        rest = [0, 2, 3]
        check_verify([t[rest] for t in (path, count, token)], [x[0][r] for r in rest], [x[1][r] for r in rest], x[2][rest], x[3][rest], x[4][rest])
    parents = [list(r) for r in x[0]]
    parents[2] = [-2] * N                       # padding
    path, count, token = verify(LL, parents, [[99] * N if r == 2 else t for r, t in enumerate(x[1])], *x[2:])
    assert LL.device_error() == 0 and count[2] == 0 and token[2] == -1 and path[2].tolist() == [-1] * N


def test_verify_offsets_past_32_bits(LL):
    n, N, V = 3, 40, 2 ** 25
    probs = torch.zeros(n, N, V, dtype=torch.bfloat16, device="cuda")      # 8 GB
    probs[:, :, V - 5] = 0.25
    probs[:, :, V - 3] = 0.75
    parents = [[-1] + list(range(N - 1))] * n
    tokens = [[0] + [V - 5] * (N - 1)] * n
    u = torch.zeros(n, N)
    u[0, 0], u[1, 0], u[2, 7] = 0.2, 0.3, 0.5
    path, count, token = LL.loglinear_tree_verify(i32(parents), i32(tokens), probs, u.cuda())
    assert count.tolist() == [N, N, 7] and token.tolist() == [V - 5, V - 3, V - 3]


# ---------------------------------------------------------------- the round

@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("drawn", [True, False])
def test_rounds(LL, graph, drawn):
    """Tree, verification and acceptance, round after round from an empty cache (one row idle), eager
    and as one captured graph: every output against the definition over what was accepted."""
    n, N, H, Hqk, dk, dv, V, M = 3, 10, 2, 1, 32, 16, 50, 4
    rounds = 70
    cache = poison(LL.LogLinearCache.empty(4, 12, H, dk, dv, M, Hqk=Hqk))
    slots, pos = i32([2, -1, 0]), i32([0, 0, 0])
    g = torch.Generator().manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731

    def inputs(i):
        parents, tokens, probs, u, draft = drafts(n, N, V, "f32", drawn, seed=100 + i)
        x = dict(q=(rand(n, N, Hqk, dk) / 6).bfloat16(), k=(rand(n, N, Hqk, dk) / 6).bfloat16(), v=rand(n, N, H, dv).bfloat16(),
                 log_a=-0.1 * torch.rand(n, N, H, generator=g), lam=torch.rand(n, N, H, M + 7, generator=g))
        return dict(x, parents=torch.tensor(parents, dtype=torch.int32), tokens=torch.tensor(tokens, dtype=torch.int32), probs=probs, u=u,
                    **({"draft": draft} if drawn else {}))

    st = {k: v.cuda() for k, v in inputs(0).items()}
    out = torch.zeros(n, N, H, dv).cuda()
    res = {}

    def once():
        LL.loglinear_cache_tree(cache, slots, pos, st["parents"], st["q"], st["k"], st["v"], st["log_a"], st["lam"], out=out)
        res["path"], res["count"], res["token"] = LL.loglinear_tree_verify(st["parents"], st["tokens"], st["probs"], st["u"], draft=st.get("draft"))
        res["new"] = LL.loglinear_cache_accept(cache, slots, pos, res["path"], st["k"], st["v"], st["log_a"])
        pos.copy_(torch.where(slots >= 0, res["new"], pos))

    if graph:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            once()
    ctx = [{"k": torch.zeros(0, Hqk, dk), "v": torch.zeros(0, H, dv), "log_a": torch.zeros(0, H)} for _ in range(n)]
    for i in range(rounds):
        host = inputs(i)
        for k, v in host.items():
            st[k].copy_(v)
        gr.replay() if graph else once()
        check_verify([res[k] for k in ("path", "count", "token")], host["parents"].tolist(), host["tokens"].tolist(), host["probs"], host["u"], host.get("draft"))
        for r in (0, 2):
            tree = {k: host[k][r].float() for k in ("q", "k", "v", "log_a", "lam")}
            check(out[r].cpu(), oracle.tree_attention(ctx[r], tree, host["parents"][r].tolist()), True)
            path = [p for p in res["path"][r].tolist() if p >= 0]
            ctx[r] = {k: torch.cat([ctx[r][k], tree[k][path]]) for k in ctx[r]}
        assert pos.tolist() == [len(ctx[0]["v"]), 0, len(ctx[2]["v"])]
    assert cache.error() == 0 and LL.device_error() == 0
    assert min(len(ctx[0]["v"]), len(ctx[2]["v"])) > 64
    invariants(cache, {2: len(ctx[0]["v"]), 0: len(ctx[2]["v"])})


def test_side_stream(LL):
    pos, N = [70, 126], 5
    cache, slots, ctx, tree, x = contexts(LL, pos, N, 2, 1, 32, 16, "bf16", True)
    twin = LL.LogLinearCache(*snapshot(cache))
    parents, paths = parents_of(2, N, "tree"), i32([[0, 1, -1], [0, 2, 3]])
    y = drafts(4, 6, 999, "f32", True)
    y = (i32(y[0]), i32(y[1]), y[2].cuda(), y[3].cuda(), y[4].cuda())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for c, stream in ((twin, side), (cache, None)):
        a = LL.loglinear_cache_tree(c, i32(slots), i32(pos), i32(parents), x["q"], x["k"], x["v"], x["log_a"], x["lam"], stream=stream)
        b = LL.loglinear_cache_accept(c, i32(slots), i32(pos), paths, x["k"], x["v"], x["log_a"], stream=stream)
        d = LL.loglinear_tree_verify(*y[:4], draft=y[4], stream=stream)
        if stream is not None:
            stream.synchronize()
        got.append((a, b, *d))
    live = torch.tensor(parents) != -2
    assert torch.equal(got[0][0][live], got[1][0][live])
    assert all(torch.equal(p, q) for p, q in zip(got[0][1:], got[1][1:]))
    assert same(snapshot(twin)[:3], snapshot(cache)[:3])
