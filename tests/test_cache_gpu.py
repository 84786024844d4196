"""The paged decode cache on the GPU: decoding from it against the definition and the dense
decode step in fp64, and the operators on its pages.

fp32 tokens: sums of up to a few hundred products of fp32 values, each decay off by at most a
few 2^-24, so rel-L2 stays below 1e-5 (TOL_F32); bf16 tokens are exact inputs, so the same
bound holds for fp32 outputs, and bf16 outputs add half a step, 2^-8 of each value.
"""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from tests.helpers import TOL_F32, per_head_qk, rel_l2, to64

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def LL():
    import log_linear_attention_fwd_gb300 as m
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def check(got, want):
    if got.dtype == torch.float32:
        assert rel_l2(got, want) <= TOL_F32, rel_l2(got, want)
    else:
        rms = float(np.sqrt(np.mean(np.square(want))))
        off = np.abs(to64(got) - want) - (2.0 ** -8 * np.abs(want) + TOL_F32 * rms)
        assert off.max() <= 0, off.max()


def poison(cache):
    """What a new cache does not define is NaN, so that any read of it shows."""
    for t in (cache.pages, cache.win_k, cache.win_v, cache.win_log_a, cache.page_log):
        t.fill_(float("nan"))
    return cache


def token(x, rows, at):
    """The tokens `at` (one per row) of sequences `rows` of forward inputs, on the GPU."""
    pick = lambda t: torch.stack([t[r, p] for r, p in zip(rows, at)]).cuda()  # noqa: E731
    return {n: None if t is None else pick(t) for n, t in x.items()}


def invariants(cache, live_rows):
    """live_rows: {slot: positions}.  Reference counts and tables fit the positions."""
    table, count = cache.page_table.cpu(), cache.refcount.cpu()
    seen = torch.zeros_like(count)
    for e in table[table >= 0].tolist():
        seen[e] += 1
    assert torch.equal(seen, count)
    for slot, n in live_rows.items():
        for m in range(cache.levels):
            if n >> 6 >> m & 1:
                assert table[slot, m] >= 0, (slot, m)


def decode(LL, cache, x, slots, start, steps, out_dtype=None, reserve=True):
    """Sequences start at different positions and go on together; returns out per step."""
    outs, pos = [], list(start)
    s = i32(slots)
    for _ in range(steps):
        d = token(x, range(len(slots)), pos)
        p = i32(pos)
        if reserve:
            LL.loglinear_cache_reserve(cache, s, p)
        outs.append(LL.loglinear_cache_step(cache, s, p, d["q"], d["k"], d["v"], d["log_a"],
                                            d["lam"], out_dtype=out_dtype))
        pos = [n + 1 for n in pos]
    return torch.stack(outs, 1), pos


@pytest.mark.parametrize("dtype,decay", [("f32", True), ("bf16", True), ("f32", False)])
@pytest.mark.parametrize("H,Hqk,dk,dv", [(2, 2, 16, 8), (4, 2, 33, 20), (3, 1, 128, 128),
                                         (1, 1, 1, 4), (2, 2, 96, 36), (6, 3, 64, 64)])
def test_decode_from_empty(LL, H, Hqk, dk, dv, dtype, decay):
    """Three blocks from nothing: every output row against the definition."""
    T, M = 200, 3
    cfg = W.FwdConfig("c", 2, H, T, dk, dv, 16, M + 7, dtype, decay, "softplus", seed=21, Hqk=Hqk)
    x = W.make_fwd_inputs(cfg)
    y = per_head_qk(x)
    want = oracle.forward_direct(y["q"], y["k"], y["v"], y["log_a"], y["lam"])
    cache = poison(LL.LogLinearCache.empty(4, 5, H, dk, dv, M, Hqk=Hqk, dtype=DT[dtype]))
    got, pos = decode(LL, cache, x, [3, 1], [0, 0], T, out_dtype=torch.float32)
    check(got.cpu(), want)
    got16, _ = decode(LL, LL.LogLinearCache.empty(4, 5, H, dk, dv, M, Hqk=Hqk, dtype=DT[dtype]),
                      x, [0, 2], [0, 0], 70, out_dtype=torch.bfloat16)
    check(got16.cpu(), want[:, :70])
    invariants(cache, {3: T, 1: T})
    assert cache.error() == 0


def dense_inputs(T, n, H, dk, dv, L, seed, dtype="f32", Hqk=None):
    """n sequences: dense states at T - 1 by the bucket definition, and tokens from T - 64 on."""
    rng = np.random.default_rng(seed)
    S = np.zeros((n, H, L, dk, dv))
    for lv in range(L):
        if (T > 0 and lv == 0) or (lv > 0 and T > 0 and (T - 1) >> (lv - 1) & 1):
            S[:, :, lv] = rng.normal(size=(n, H, dk, dv)) * 0.5
    g = torch.Generator().manual_seed(seed)
    Hqk = Hqk or H
    tok = lambda steps: dict(  # noqa: E731
        q=torch.randn(n, steps, Hqk, dk, generator=g).to(DT[dtype]),
        k=(torch.randn(n, steps, Hqk, dk, generator=g) / dk ** 0.5).to(DT[dtype]),
        v=torch.randn(n, steps, H, dv, generator=g).to(DT[dtype]),
        log_a=-0.1 * torch.rand(n, steps, H, generator=g), lam=torch.rand(n, steps, H, L, generator=g))
    return torch.from_numpy(S).float(), tok


def block_states(S, tok, T):
    """Puts the true levels inside the last block into S, from the prompt's tokens."""
    r = T % 64
    n, H, L, dk, dv = S.shape
    Hqk = tok["k"].shape[2]
    for b in range(n):
        for h in range(H):
            hq = h // (H // Hqk)
            k, v = to64(tok["k"][b, :, hq])[-r:], to64(tok["v"][b, :, h])[-r:]
            la = to64(tok["log_a"][b, :, h])[-r:]
            s = oracle.states_from_buckets(k, v, la, r - 1, 7)
            S[b, h, :7] = torch.from_numpy(np.asarray(s)[:7]).float()
    return S


@pytest.mark.parametrize("T", [0, 1, 2, 63, 64, 65, 127, 128, 192, 4095, 4096, 12288, 12345, 16383])
def test_load_then_decode(LL, T):
    """A prompt's dense states go in, 70 steps follow (over one or two block ends), against the
    dense step in fp64; then the states come out again."""
    n, H, dk, dv, M = 2, 2, 16, 8, 9
    L = M + 7
    S, tok = dense_inputs(T, n, H, dk, dv, L, seed=T)
    prompt = tok(64)
    if T % 64:
        S = block_states(S, prompt, T)
    x = tok(70)
    cache = poison(LL.LogLinearCache.empty(3, 24, H, dk, dv, M, dtype=torch.float32))
    slots = i32([2, 0])
    c = lambda t: t.cuda()  # noqa: E731
    LL.loglinear_cache_load(cache, slots, T, c(S), c(prompt["k"]), c(prompt["v"]), c(prompt["log_a"]))
    ref = S.double().numpy()
    for i in range(70):
        t = T + i
        p = i32([t, t])
        LL.loglinear_cache_reserve(cache, slots, p)
        a = {k: v[:, i].contiguous() for k, v in x.items()}
        out = LL.loglinear_cache_step(cache, slots, p, *(c(a[k]) for k in ("q", "k", "v", "log_a", "lam")))
        ref, want = oracle.decode_step(ref, a["q"], a["k"], a["v"], a["log_a"], a["lam"], t)
        check(out.cpu(), want)
        if i in (0, 5, 69) or (t + 1) % 64 == 0:
            got = LL.loglinear_cache_store(cache, slots, p + 1).cpu()
            if (t + 1) % 64:
                check(got, ref)
            else:  # the levels that the next step merges come as their sum
                l = oracle.lssb(t + 1)
                check(got[:, :, l], ref[:, :, :l + 1].sum(2))
                assert torch.all(got[:, :, :l] == 0)
                if l + 1 < L:
                    check(got[:, :, l + 1:], ref[:, :, l + 1:]) if np.any(ref[:, :, l + 1:]) else None
    invariants(cache, {2: T + 70, 0: T + 70})
    assert cache.error() == 0


@pytest.mark.parametrize("decay", [True, False])
def test_prefill_load_decode_store(LL, decay):
    """The whole way: prefill, load, decode in the cache, store, dense decode; fp32 and bf16."""
    for dtype in ("f32", "bf16"):
        T, steps, M = 150, 60, 3
        cfg = W.FwdConfig("c", 2, 2, T + steps, 32, 16, 16, M + 7, dtype, decay, "softplus", seed=5)
        x = W.make_fwd_inputs(cfg)
        want = oracle.forward_direct(x["q"], x["k"], x["v"], x["log_a"], x["lam"])
        d = {k: None if v is None else v.cuda() for k, v in x.items()}
        cut = {k: None if v is None else v[:, :T].contiguous() for k, v in d.items()}
        _, state = LL.loglinear_prefill(cut["q"], cut["k"], cut["v"], cut["log_a"], cut["lam"], 16)
        cache = poison(LL.LogLinearCache.empty(2, 6, 2, 32, 16, M, dtype=DT[dtype]))
        tail = lambda t: None if t is None else t[:, T - 40:T]  # noqa: E731  strided views
        LL.loglinear_cache_load(cache, i32([0, 1]), T, state, tail(d["k"]), tail(d["v"]), tail(d["log_a"]))
        got, pos = decode(LL, cache, x, [0, 1], [T, T], 30, out_dtype=torch.float32)
        check(got.cpu(), want[:, T:T + 30])
        dense = LL.loglinear_cache_store(cache, i32([0, 1]), i32(pos))
        for t in range(T + 30, T + steps):
            a = {k: None if v is None else v[:, t].contiguous() for k, v in d.items()}
            o = LL.loglinear_decode_step(dense, a["q"], a["k"], a["v"], a["log_a"], a["lam"], t,
                                         out_dtype=torch.float32)
            check(o.cpu(), want[:, t])


def test_sequences_at_positions_of_their_own(LL):
    """Staggered starts, rows that pause, padding rows: each row as if it were alone."""
    H, dk, dv, M, T = 2, 16, 8, 3, 150
    cfg = W.FwdConfig("c", 4, H, T, dk, dv, 16, M + 7, "f32", True, "softplus", seed=3)
    x = W.make_fwd_inputs(cfg)
    want = oracle.forward_direct(x["q"], x["k"], x["v"], x["log_a"], x["lam"])
    cache = poison(LL.LogLinearCache.empty(6, 9, H, dk, dv, M, dtype=torch.float32))
    slots, pos = [5, 0, 3, 2], [0, 0, 0, 0]
    rng = np.random.default_rng(0)
    while min(pos) < T:
        act = [i for i in range(4) if pos[i] < T and rng.random() < 0.4 + 0.15 * i]
        if not act:
            continue
        rows = list(rng.permutation(act)) + [act[0]]          # the last row is padding
        d = token(x, rows, [pos[i] for i in rows])
        s = i32([slots[i] for i in rows[:-1]] + [-1])
        p = i32([pos[i] for i in rows])
        out = torch.full((len(rows), H, dv), 7.0).cuda()
        LL.loglinear_cache_reserve(cache, s, p)
        LL.loglinear_cache_step(cache, s, p, d["q"], d["k"], d["v"], d["log_a"], d["lam"], out=out)
        assert torch.all(out[-1] == 7)
        check(out[:-1].cpu(), np.stack([want[i, pos[i]] for i in rows[:-1]]))
        for i in rows[:-1]:
            pos[i] += 1
    invariants(cache, {s: T for s in slots})
    assert cache.error() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,H,Hqk,dk,dv", [(70, 3, 3, 16, 8), (40, 4, 2, 33, 20), (26, 6, 1, 128, 128),
                                           (160, 1, 1, 64, 36), (400, 2, 1, 8, 4)])
def test_batches_of_more_items_than_sms(LL, n, H, Hqk, dk, dv, dtype):
    """Rows at positions all over, block ends among them, with rows that are padding or cannot be
    served in between; three steps, each against the dense step in fp64, and the states after."""
    M = 8
    L = M + 7
    rng = np.random.default_rng(n)
    cache = poison(LL.LogLinearCache.empty(n, 5 * n, H, dk, dv, M, Hqk=Hqk, dtype=DT[dtype]))
    kinds = [0, 1, 62, 63, 64, 126, 127, 4095, 4094, 8190, 12345, 61] + rng.integers(0, 16000, 6).tolist()
    T = [kinds[i % len(kinds)] for i in range(n)]
    slots = rng.permutation(n)
    ref = np.zeros((n, H, L, dk, dv))
    for t0 in sorted(set(T)):
        rows = [i for i in range(n) if T[i] == t0]
        S, tok = dense_inputs(t0, len(rows), H, dk, dv, L, seed=t0, dtype=dtype, Hqk=Hqk)
        prompt = tok(64)
        if t0 % 64:
            S = block_states(S, prompt, t0)
        c = {k: v.cuda() for k, v in prompt.items()}
        LL.loglinear_cache_load(cache, i32(slots[rows]), t0, S.cuda(), c["k"], c["v"], c["log_a"])
        ref[rows] = S.double().numpy()
    assert cache.error() == 0
    _, tok = dense_inputs(1, n, H, dk, dv, L, seed=3, dtype=dtype, Hqk=Hqk)
    x = tok(3)
    s = i32(slots)
    idle = [3, n - 1]
    s_idle = s.clone()
    s_idle[idle[0]], s_idle[idle[1]] = -1, n + 5
    for i in range(3):
        p = i32([t + i for t in T])
        a = {k: v[:, i].contiguous().cuda() for k, v in x.items()}
        args = (a["q"], a["k"], a["v"], a["log_a"], a["lam"])
        LL.loglinear_cache_reserve(cache, s, p)
        out = torch.full((n, H, dv), 7.0).cuda()
        LL.loglinear_cache_step(cache, s_idle, p, *args, out=out)
        assert torch.all(out[idle] == 7) and cache.error() == LL.CACHE_ERR_SLOT
        LL.loglinear_cache_step(cache, s, p, *args, out=out)
        assert cache.error() == 0
        y = {k: to64(v[:, i]) for k, v in x.items()}
        y["q"], y["k"] = (np.repeat(y[k], H // Hqk, axis=1) for k in ("q", "k"))
        for b in range(n):
            new, want = oracle.decode_step(ref[b:b + 1], *(y[k][b:b + 1] for k in ("q", "k", "v", "log_a", "lam")), T[b] + i)
            ref[b] = new[0]
            check(out[b].cpu(), want[0])
    got = LL.loglinear_cache_store(cache, s, i32([t + 3 for t in T])).cpu()
    for b in range(n):
        if (T[b] + 3) % 64:
            check(got[b], ref[b])
    invariants(cache, {int(slots[b]): T[b] + 3 for b in range(n)})


def filled(LL, seed=0, n=3, T=(100, 200, 320), spare=12, dtype="f32", M=4, more=80):
    """A cache with n sequences decoded from nothing, and their inputs."""
    H, dk, dv = 2, 16, 8
    cfg = W.FwdConfig("c", n, H, max(T) + more, dk, dv, 16, M + 7, dtype, True, "softplus", seed=seed)
    x = W.make_fwd_inputs(cfg)
    cache = poison(LL.LogLinearCache.empty(8, 3 * n + spare, H, dk, dv, M, dtype=DT[dtype]))
    for i in range(n):
        one = {k: v[i:i + 1] for k, v in x.items()}
        decode(LL, cache, one, [i], [0], T[i])
    return cache, x, list(T)


def snapshot(cache):
    return [t.clone() for t in (cache.pages, cache.page_table, cache.refcount, cache.win_k,
                                cache.win_v, cache.win_log_a, cache.page_log, cache.page_from)]


def same(a, b):
    return all(torch.equal(x.nan_to_num(5.0), y.nan_to_num(5.0)) for x, y in zip(a, b))


@pytest.mark.parametrize("at", [(70, 130, 300), (63, 127, 191), (64, 128, 256)])
def test_a_step_can_be_repeated(LL, at):
    """Reservation and step at the same positions twice: the same outputs, the same cache."""
    cache, x, _ = filled(LL, T=at)
    d = token(x, range(3), at)
    s, p = i32([0, 1, 2]), i32(at)
    run = lambda: (LL.loglinear_cache_reserve(cache, s, p), LL.loglinear_cache_step(  # noqa: E731
        cache, s, p, d["q"], d["k"], d["v"], d["log_a"], d["lam"]))[1]
    one = run()
    snap = snapshot(cache)
    two = run()
    assert torch.equal(one, two) and same(snap, snapshot(cache)) and cache.error() == 0


def test_fork(LL):
    """Forks decode as their source would with the same tokens, and apart from it with others;
    shared pages outlive the source."""
    cache, x, T = filled(LL)
    H, dk, dv = 2, 16, 8
    src, dst = i32([2, 1, 2]), i32([5, 6, 7])
    before = cache.refcount.clone()
    LL.loglinear_cache_fork(cache, src, dst, i32([T[2], T[1], T[2]]))
    assert int(cache.refcount.sum()) == int(before.sum()) + 2 * bin(T[2] >> 6).count("1") + bin(T[1] >> 6).count("1")
    assert torch.equal(cache.refcount > 0, before > 0)
    want = oracle.forward_direct(x["q"], x["k"], x["v"], x["log_a"], x["lam"])
    # source 2 and fork 5 take the same tokens, fork 7 another sequence's
    other = {k: v.clone() for k, v in x.items()}
    for k in other:
        other[k][2, T[2]:] = other[k][0, :other[k].shape[1] - T[2]]
    want7 = oracle.forward_direct(*(other[k][2:] for k in ("q", "k", "v", "log_a", "lam")))
    both = {k: torch.stack([x[k][2], x[k][2], other[k][2], x[k][1]]) for k in x}
    got, pos = decode(LL, cache, both, [2, 5, 7, 6], [T[2], T[2], T[2], T[1]], 30)
    check(got[0].cpu(), want[2, T[2]:T[2] + 30])
    assert torch.equal(got[0], got[1])
    check(got[2].cpu(), want7[0, T[2]:T[2] + 30])
    check(got[3].cpu(), want[1, T[1]:T[1] + 30])
    LL.loglinear_cache_free(cache, i32([2, -1, 5]))
    more, _ = decode(LL, cache, {k: v[2:] for k, v in both.items()}, [7, 6], pos[2:], 40)
    check(more[0].cpu(), want7[0, T[2] + 30:T[2] + 70])
    check(more[1].cpu(), want[1, T[1] + 30:T[1] + 70])
    invariants(cache, {7: T[2] + 70, 6: T[1] + 70, 0: T[0]})
    LL.loglinear_cache_free(cache, i32([0, 1, 6, 7]))
    assert int(cache.refcount.sum()) == 0 and torch.all(cache.page_table == -1)
    assert cache.error() == 0


def test_a_fold_never_writes_a_shared_page(LL):
    """Pages left over from earlier positions (no reservation at the blocks' first positions) may
    still be a fork's live ones: the reservation at the block's end replaces them, and a step
    without it is refused."""
    cache, x, _ = filled(LL, n=1, T=(64 + 10,), more=160)  # page of level 0 is live in slot 0
    LL.loglinear_cache_fork(cache, i32([0, 0]), i32([3, 4]), i32([74, 74]))
    want = oracle.forward_direct(x["q"], x["k"], x["v"], x["log_a"], x["lam"])
    pos = 74
    one = {k: v[:1] for k, v in x.items()}
    while pos < 191:                                       # slots 0 and 4 go on; slot 3 stays at 74
        got, (pos, _) = decode(LL, cache, {k: torch.cat([v, v]) for k, v in one.items()}, [0, 4], [pos, pos], 1,
                               reserve=pos in (127,))
        check(got[:, 0].cpu(), want[[0, 0], pos - 1])
    assert cache.error() == 0 and (cache.page_table[[0, 3, 4], 0] == cache.page_table[0, 0]).all()
    snap = snapshot(cache)
    d = token(one, [0], [191])                             # position 191 folds into level 0
    LL.loglinear_cache_step(cache, i32([0]), i32([191]), d["q"], d["k"], d["v"], d["log_a"], d["lam"])
    assert cache.error() == LL.CACHE_ERR_MISSING and same(snap, snapshot(cache))
    got, _ = decode(LL, cache, {k: torch.cat([v, v]) for k, v in one.items()}, [0, 4], [191, 191], 40)
    check(got.cpu(), want[[0, 0], 191:231])
    invariants(cache, {0: 231, 4: 231, 3: 74})
    got, _ = decode(LL, cache, one, [3], [74], 40)         # and the fork that stayed is whole
    check(got.cpu(), want[:1, 74:114])
    assert cache.error() == 0


def test_fork_replaces_its_target(LL):
    cache, x, T = filled(LL)
    LL.loglinear_cache_fork(cache, i32([1]), i32([2]), i32([T[1]]))
    invariants(cache, {2: T[1], 1: T[1], 0: T[0]})
    LL.loglinear_cache_fork(cache, i32([1]), i32([2]), i32([T[1]]))   # again, onto itself's copy
    invariants(cache, {2: T[1], 1: T[1], 0: T[0]})
    want = oracle.forward_direct(x["q"], x["k"], x["v"], x["log_a"], x["lam"])
    got, _ = decode(LL, cache, {k: v[1:2] for k, v in x.items()}, [2], [T[1]], 10)
    check(got[0].cpu(), want[1, T[1]:T[1] + 10])


def test_compact(LL):
    """Holes are filled from above in order; decoding goes on bit for bit, forks included."""
    cache, x, T = filled(LL, T=(100, 250, 340), spare=6)
    LL.loglinear_cache_fork(cache, i32([2]), i32([4]), i32([T[2]]))
    LL.loglinear_cache_free(cache, i32([0, 1]))
    twin = LL.LogLinearCache(*[t.clone() for t in (cache.pages, cache.page_table, cache.refcount, cache.win_k, cache.win_v,
                                                   cache.win_log_a, cache.page_log, cache.page_from)])
    used = (cache.refcount > 0).nonzero()[:, 0].tolist()
    live = LL.loglinear_cache_compact(cache)
    n = int(live)
    assert n == len(used) and torch.all(cache.refcount[:n] == 2) and torch.all(cache.refcount[n:] == 0)
    holes = [p for p in range(n) if p not in used]
    high = [p for p in used if p >= n]
    for h, p in zip(holes, high):
        assert torch.equal(cache.pages[h], twin.pages[p])
    invariants(cache, {2: T[2], 4: T[2]})
    again = LL.loglinear_cache_compact(cache)
    assert int(again) == n
    both = {k: v[2:] for k, v in x.items()}
    a, _ = decode(LL, cache, both, [2], [T[2]], 50)
    b, _ = decode(LL, twin, both, [2], [T[2]], 50)
    assert torch.equal(a, b) and cache.error() == 0
    LL.loglinear_cache_free(cache, i32([2, 4]))
    assert int(LL.loglinear_cache_compact(cache)) == 0


def test_pages_are_taken_lowest_first(LL):
    cache = LL.LogLinearCache.empty(6, 2100, 1, 4, 4, 5, dtype=torch.float32)
    cache.refcount[:2000] = 1
    cache.refcount[[3, 17, 1030, 1031]] = 0
    cache.refcount[2001] = 1
    T = 64 * 7
    S = torch.randn(3, 1, 16, 4, 4).cuda()
    k = torch.zeros(3, 1, 1, 4).cuda()
    LL.loglinear_cache_load(cache, i32([4, -1, 1]), T, S, k, k, None)
    assert cache.page_table[4, :3].tolist() == [3, 17, 1030]
    assert cache.page_table[1, :3].tolist() == [1031, 2000, 2002]
    assert cache.error() == 0


def test_more_rows_than_a_plan_has_threads(LL):
    """1500 rows at once (their owners go through memory) against two calls of fewer rows."""
    n, H, d, M = 1500, 2, 8, 3
    g = torch.Generator().manual_seed(5)
    perm = torch.randperm(1600, generator=g)[:n].to(torch.int32)
    perm[torch.randperm(n, generator=g)[:40]] = -1
    pos = torch.full((n,), 63, dtype=torch.int32)
    pos[torch.randperm(n, generator=g)[:300]] = 62
    perm, pos = perm.cuda(), pos.cuda()
    S = torch.randn(n, H, M + 7, d, d, generator=g).cuda()
    k, v = torch.randn(n, 63, H, d, generator=g).cuda(), torch.randn(n, 63, H, d, generator=g).cuda()
    la, lam = -torch.rand(n, 63, H, generator=g).cuda(), torch.rand(n, H, M + 7, generator=g).cuda()
    parts = {1: [slice(0, n)], 2: [slice(0, 700), slice(700, n)]}
    got = {}
    for calls in parts:
        cache = poison(LL.LogLinearCache.empty(1600, 1400, H, d, d, M, dtype=torch.float32))
        out = torch.full((n, H, d), 7.0).cuda()
        for at in parts[calls]:
            cut = lambda t: t[at].contiguous()  # noqa: E731
            LL.loglinear_cache_load(cache, cut(perm), 62, cut(S), k[at, :62], v[at, :62], la[at, :62])
        for last in (62, 63):  # (rows at 62 are repeated)
            for at in parts[calls]:
                cut = lambda t: t[at].contiguous()  # noqa: E731
                p = torch.minimum(pos, torch.full_like(pos, last))
                LL.loglinear_cache_reserve(cache, cut(perm), cut(p))
                LL.loglinear_cache_step(cache, cut(perm), cut(p), cut(k[:, 0]), cut(k[:, 1]), cut(v[:, 0]),
                                        cut(la[:, 62]), cut(lam), out=out[at])
        assert cache.error() == 0
        got[calls] = (out, cache.page_table, cache.refcount)
        invariants(cache, {int(s): 64 for s, p in zip(perm, pos) if s >= 0 and p == 63})
    for a, b in zip(got[1], got[2]):
        assert torch.equal(a, b)
    assert torch.all(got[1][0][perm < 0] == 7)
    twice = perm.clone()
    twice[1400] = perm[perm >= 0][3]
    LL.loglinear_cache_reserve(cache, twice, pos)
    assert cache.error() == LL.CACHE_ERR_SLOT


def test_pool_runs_out(LL):
    """A row that gets no page is left out, the others go on; nothing is written astray."""
    H, dk, dv, M = 2, 16, 8, 3
    cfg = W.FwdConfig("c", 3, H, 70, dk, dv, 16, M + 7, "f32", True, "softplus", seed=3)
    x = W.make_fwd_inputs(cfg)
    want = oracle.forward_direct(x["q"], x["k"], x["v"], x["log_a"], x["lam"])
    cache = LL.LogLinearCache.empty(3, 2, H, dk, dv, M, dtype=torch.float32)
    decode(LL, cache, x, [0, 1, 2], [0, 0, 0], 63)
    s, p = i32([0, 1, 2]), i32([63] * 3)
    LL.loglinear_cache_reserve(cache, s, p)
    assert cache.error() == LL.CACHE_ERR_PAGES and cache.error() == 0
    d = token(x, range(3), [63] * 3)
    out = torch.full((3, H, dv), 7.0).cuda()
    LL.loglinear_cache_step(cache, s, p, d["q"], d["k"], d["v"], d["log_a"], d["lam"], out=out)
    assert cache.error() == LL.CACHE_ERR_MISSING
    check(out[:2].cpu(), want[:2, 63])
    assert torch.all(out[2] == 7)
    # room is made, and the row catches up
    LL.loglinear_cache_free(cache, i32([0]))
    LL.loglinear_cache_reserve(cache, i32([2]), i32([63]))
    got, _ = decode(LL, cache, {k: v[2:] for k, v in x.items()}, [2], [63], 5)
    check(got[0].cpu(), want[2, 63:68])
    assert cache.error() == 0


def test_rows_that_cannot_be_served(LL):
    """Slots out of range or given twice, positions outside the cache, pages not there: those
    rows raise the error word and change nothing, the others are served."""
    cache, x, T = filled(LL)
    M, want = cache.levels, oracle.forward_direct(x["q"], x["k"], x["v"], x["log_a"], x["lam"])
    rows = [0, 1, 1, 2, 2, 0]
    slots, pos = [0, 1, 1, 8, -3, 4], [T[0], T[1], T[1], 0, 0, 64]
    d = token(x, rows, [T[0], T[1], T[1], 0, 0, 64])
    snap = snapshot(cache)
    out = torch.full((6, 2, 8), 7.0).cuda()
    args = (d["q"], d["k"], d["v"], d["log_a"], d["lam"])
    LL.loglinear_cache_step(cache, i32(slots), i32(pos), *args, out=out)
    assert cache.error() == LL.CACHE_ERR_SLOT | LL.CACHE_ERR_MISSING
    check(out[:2].cpu(), np.stack([want[0, T[0]], want[1, T[1]]]))
    assert torch.all(out[2:] == 7)
    assert torch.equal(cache.page_table, snap[1]) and torch.equal(cache.pages.nan_to_num(5.0), snap[0].nan_to_num(5.0))
    assert torch.equal(cache.win_k[2:].nan_to_num(5.0), snap[3][2:].nan_to_num(5.0))
    top = 64 * 2 ** M - 1
    snap = snapshot(cache)
    for bad in (-1, top, top + 5, 2 ** 31 - 1):
        d = token(x, [0], [0])
        LL.loglinear_cache_step(cache, i32([0]), i32([bad]), d["q"], d["k"], d["v"], d["log_a"], d["lam"])
        assert cache.error() == LL.CACHE_ERR_POSITION
        LL.loglinear_cache_reserve(cache, i32([0]), i32([bad]))
        assert cache.error() == LL.CACHE_ERR_POSITION
    for call in (lambda: LL.loglinear_cache_fork(cache, i32([0, 1]), i32([5, 5]), i32([T[0], T[1]])),   # target twice
                 lambda: LL.loglinear_cache_free(cache, i32([5, 9]))):
        call()
        assert cache.error() == LL.CACHE_ERR_SLOT
    assert same(snap[1:3], snapshot(cache)[1:3])
    LL.loglinear_cache_fork(cache, i32([0, 1, 9]), i32([1, 4, 5]), i32([T[0], T[1], 0]))  # a source that is a target
    assert cache.error() == LL.CACHE_ERR_SLOT
    invariants(cache, {0: T[0], 1: T[0], 2: T[2]})
    LL.loglinear_cache_reserve(cache, i32([2, 2]), i32([T[2], T[2]]))
    assert cache.error() == LL.CACHE_ERR_SLOT
    cache.page_table[2, 0], cache.page_table[2, 2] = 10 ** 6, -7    # a table that was overwritten
    d = token(x, [2], [T[2]])
    LL.loglinear_cache_step(cache, i32([2]), i32([T[2]]), d["q"], d["k"], d["v"], d["log_a"], d["lam"])
    st = torch.full((1, 2, M + 7, 16, 8), 3.0).cuda()
    LL.loglinear_cache_store(cache, i32([2]), i32([T[2]]), st)
    assert cache.error() == LL.CACHE_ERR_MISSING


def test_resets_and_extreme_decays(LL):
    """log a of -inf (a = 0) and the type's lowest value drop all that came before, pages too."""
    H, dk, dv, M, T = 1, 8, 4, 3, 260
    cfg = W.FwdConfig("c", 1, H, T, dk, dv, 16, M + 7, "f32", True, "softplus", seed=3)
    x = W.make_fwd_inputs(cfg)
    x["log_a"][0, 30], x["log_a"][0, 100] = -float("inf"), torch.finfo(torch.float32).min
    x["log_a"][0, 200], x["log_a"][0, 201] = -float("inf"), 0.0
    y = {k: v.clone() for k, v in x.items()}
    y["log_a"] = y["log_a"].clamp(min=-1e4)      # the same decays, without inf - inf in the oracle
    want = oracle.forward_direct(y["q"], y["k"], y["v"], y["log_a"], y["lam"])
    cache = LL.LogLinearCache.empty(1, 6, H, dk, dv, M, dtype=torch.float32)
    got, _ = decode(LL, cache, x, [0], [0], T)
    check(got.cpu(), want)


def test_graph_replay(LL):
    """Reservation and step captured once; positions and tokens change in place."""
    H, dk, dv, M, T = 2, 16, 8, 3, 140
    cfg = W.FwdConfig("c", 2, H, T, dk, dv, 16, M + 7, "bf16", True, "softplus", seed=3)
    x = W.make_fwd_inputs(cfg)
    caches = [poison(LL.LogLinearCache.empty(2, 6, H, dk, dv, M)) for _ in range(2)]
    eager, _ = decode(LL, caches[0], x, [1, 0], [0, 0], T)
    s, p = i32([1, 0]), i32([0, 0])
    d = token(x, [0, 1], [0, 0])
    out = torch.empty(2, H, dv, dtype=torch.bfloat16).cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        LL.loglinear_cache_reserve(caches[1], s, p)
        LL.loglinear_cache_step(caches[1], s, p, d["q"], d["k"], d["v"], d["log_a"], d["lam"], out=out)
    for t in range(T):
        p.fill_(t)
        for k, v in token(x, [0, 1], [t, t]).items():
            d[k].copy_(v)
        g.replay()
        assert torch.equal(out, eager[:, t])
    assert same(snapshot(caches[0])[:3], snapshot(caches[1])[:3]) and caches[1].error() == 0


def test_side_stream(LL):
    cache, x, T = filled(LL)
    twin = LL.LogLinearCache(*snapshot(cache))
    d = token(x, range(3), T)
    s, p = i32([0, 1, 2]), i32(T)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = LL.loglinear_cache_step(twin, s, p, d["q"], d["k"], d["v"], d["log_a"], d["lam"], stream=side)
    b = LL.loglinear_cache_step(cache, s, p, d["q"], d["k"], d["v"], d["log_a"], d["lam"])
    side.synchronize()
    assert torch.equal(a, b)


def test_large_pool_offsets(LL):
    """Pages whose element offsets pass 32 bits."""
    H, dk, dv, M = 16, 128, 128, 2
    n_pages = 2 ** 32 // (H * dk * dv) // 2 + 60          # 2^31 elements: 8.6 GB
    cache = LL.LogLinearCache.empty(2, n_pages, H, dk, dv, M)
    cache.refcount[:n_pages - 2] = 1
    cfg = W.FwdConfig("c", 1, H, 70, dk, dv, 16, M + 7, "bf16", True, "softplus", seed=3)
    x = W.make_fwd_inputs(cfg)
    got, _ = decode(LL, cache, x, [1], [0], 70, out_dtype=torch.float32)
    want = oracle.forward_direct(x["q"], x["k"], x["v"], x["log_a"], x["lam"])
    check(got.cpu(), want)
    assert cache.page_table[1].tolist() == [n_pages - 2, -1] and cache.error() == 0
    cache.refcount[:n_pages - 2] = 0
    assert int(LL.loglinear_cache_compact(cache)) == 1 and cache.page_table[1, 0] == 0
    dense = LL.loglinear_cache_store(cache, i32([1]), i32([70]))
    k, v, la = (to64(x[n][0, :64, 5]) for n in ("k", "v", "log_a"))
    w = np.exp(to64(x["log_a"][0, :70, 5]).sum() - np.cumsum(la))
    check(dense[0, 5, 7].cpu(), np.einsum("s,sd,se->de", w, k, v))


@pytest.mark.parametrize("gone", [-1, 10 ** 6, -7])
def test_a_fork_without_its_sources_pages_is_left_out(LL, gone):
    """A source whose page is not there: its row's target stays as it was, pages, tokens and
    counts; so does what would be forked from that target.  The other rows are served."""
    cache, x, T = filled(LL)                                   # slot 1 holds pages 0 and 1, slot 2 pages 0 and 2
    cache.refcount[cache.page_table[1, 1]] -= 1
    cache.page_table[1, 1] = gone
    LL.loglinear_cache_fork(cache, i32([2]), i32([4]), i32([T[2]]))
    assert cache.error() == 0
    snap = snapshot(cache)
    LL.loglinear_cache_fork(cache, i32([1, 4]), i32([4, 6]), i32([T[1], T[2]]))
    assert cache.error() == LL.CACHE_ERR_MISSING | LL.CACHE_ERR_SLOT and same(snap, snapshot(cache))
    LL.loglinear_cache_fork(cache, i32([1, 0]), i32([4, 5]), i32([T[1], T[0]]))
    assert cache.error() == LL.CACHE_ERR_MISSING
    now = snapshot(cache)
    keep = [0, 1, 2, 3, 4, 6, 7]
    assert same([t[keep] for t in (snap[1], *snap[3:])], [t[keep] for t in (now[1], *now[3:])])
    snap[2][cache.page_table[0, 0]] += 1
    assert same(snap[:1] + snap[2:3], now[:1] + now[2:3])
    want = oracle.forward_direct(x["q"], x["k"], x["v"], x["log_a"], x["lam"])
    both = {k: v[[2, 0]] for k, v in x.items()}
    got, _ = decode(LL, cache, both, [4, 5], [T[2], T[0]], 40)
    check(got[0].cpu(), want[2, T[2]:T[2] + 40])
    check(got[1].cpu(), want[0, T[0]:T[0] + 40])
    assert cache.error() == 0


def test_a_store_without_its_pages_is_left_out(LL):
    """A row whose page is not there, or whose position is outside the cache, keeps its output
    whole; the others are served."""
    cache, x, T = filled(LL)
    M = cache.levels
    want = LL.loglinear_cache_store(cache, i32([0]), i32([T[0]]))
    for gone in (-1, 10 ** 6, -7):
        cache.page_table[2, 2] = gone
        st = torch.full((4, 2, M + 7, 16, 8), 3.0).cuda()
        LL.loglinear_cache_store(cache, i32([2, 0, 2, -1]), i32([T[2], T[0], T[2] - 1, 0]), st)
        assert cache.error() == LL.CACHE_ERR_MISSING
        assert torch.all(st[[0, 2, 3]] == 3) and torch.equal(st[1], want[0])   # (319 is in block 4: page 2 too)
    st = torch.full((2, 2, M + 7, 16, 8), 3.0).cuda()
    LL.loglinear_cache_store(cache, i32([0, 0]), i32([-1, T[0]]), st)
    assert cache.error() == LL.CACHE_ERR_POSITION and torch.all(st[0] == 3) and torch.equal(st[1], want[0])


@pytest.mark.parametrize("rows", [2, 90])
def test_going_back_before_the_load(LL, rows):
    """A loaded prompt's pages have decayed to its end: a position before it, in a block with
    pages, is refused by the step, the store and the fork, and changes nothing."""
    H, dk, dv, M, T = 2, 16, 8, 3, 100
    L = M + 7
    S, tok = dense_inputs(T, rows, H, dk, dv, L, seed=T)
    prompt = tok(64)
    S = block_states(S, prompt, T)
    x = tok(3)
    cache = poison(LL.LogLinearCache.empty(rows + 2, 2 * rows, H, dk, dv, M, dtype=torch.float32))
    slots = torch.arange(rows, dtype=torch.int32).cuda()
    c = lambda t: t.cuda()  # noqa: E731
    LL.loglinear_cache_load(cache, slots, T, c(S), c(prompt["k"]), c(prompt["v"]), c(prompt["log_a"]))
    arg = lambda i: [x[k][:, i].contiguous().cuda() for k in ("q", "k", "v", "log_a", "lam")]  # noqa: E731
    one = LL.loglinear_cache_step(cache, slots, torch.full_like(slots, T), *arg(0))
    LL.loglinear_cache_step(cache, slots, torch.full_like(slots, T + 1), *arg(1))
    assert cache.error() == 0
    snap = snapshot(cache)
    pos = torch.full_like(slots, T)
    pos[1] = T - 1
    out = torch.full_like(one, 7.0)
    LL.loglinear_cache_step(cache, slots, pos, *arg(0), out=out)
    assert cache.error() == LL.CACHE_ERR_POSITION and torch.all(out[1] == 7)
    assert torch.equal(out[0], one[0]) and torch.equal(out[2:], one[2:]) and same(snap, snapshot(cache))
    st = torch.full((rows, H, L, dk, dv), 3.0).cuda()
    LL.loglinear_cache_store(cache, slots, pos, st)
    assert cache.error() == LL.CACHE_ERR_POSITION and torch.all(st[1] == 3)
    check(st[0].cpu(), S[0].numpy())
    LL.loglinear_cache_fork(cache, slots[:2].contiguous(), i32([rows, rows + 1]), pos[:2].contiguous())
    assert cache.error() == LL.CACHE_ERR_POSITION
    assert cache.page_table[rows, 0] == cache.page_table[0, 0] and torch.all(cache.page_table[rows + 1] == -1)
    # in block 0 there are no pages, so any position of it may come again
    LL.loglinear_cache_load(cache, slots[:1].contiguous(), 36, c(S[:1]), c(prompt["k"][:1]), c(prompt["v"][:1]),
                            c(prompt["log_a"][:1]))
    LL.loglinear_cache_step(cache, slots[:1].contiguous(), i32([20]), *(t[:1].contiguous() for t in arg(2)))
    assert cache.error() == 0


@pytest.mark.parametrize("at", [70, 127])
def test_going_back_inside_a_block(LL, at):
    """Positions of the current block may come again with other tokens, its end among them."""
    cache, x, _ = filled(LL, n=1, T=(128,), more=60)           # block 1 has been folded
    back = {k: v.clone() for k, v in x.items()}
    g = torch.Generator().manual_seed(1)
    for k in ("q", "k", "v"):
        back[k][:, at:] = torch.randn(back[k][:, at:].shape, generator=g)
    want = oracle.forward_direct(*(back[k] for k in ("q", "k", "v", "log_a", "lam")))
    got, _ = decode(LL, cache, back, [0], [at], 188 - at)
    check(got.cpu(), want[:, at:188])
    invariants(cache, {0: 188})
    assert cache.error() == 0


def test_a_draft_across_a_blocks_end_on_a_fork(LL):
    """Drafted tokens that cross a block's end are decoded on a fork; rejected, the slot goes on
    from where it was."""
    cache, x, _ = filled(LL, n=1, T=(126,), more=60)
    draft = {k: v.clone() for k, v in x.items()}
    draft["v"][:, 126:] = draft["v"][:, :draft["v"].shape[1] - 126]
    LL.loglinear_cache_fork(cache, i32([0]), i32([5]), i32([126]))
    got, _ = decode(LL, cache, draft, [5], [126], 6)
    check(got.cpu(), oracle.forward_direct(*(draft[k] for k in ("q", "k", "v", "log_a", "lam")))[:, 126:132])
    LL.loglinear_cache_free(cache, i32([5]))
    got, _ = decode(LL, cache, x, [0], [126], 60)
    check(got.cpu(), oracle.forward_direct(*(x[k] for k in ("q", "k", "v", "log_a", "lam")))[:, 126:186])
    invariants(cache, {0: 186})
    assert cache.error() == 0


def test_fork_rows_without_a_source_are_padding(LL):
    """-1 as a source leaves the row out, as it does as a target: no error, and the target is
    free for another row."""
    cache, x, T = filled(LL)
    snap = snapshot(cache)
    LL.loglinear_cache_fork(cache, i32([-1, 1, 0, -1]), i32([5, 5, -1, -1]), i32([0, T[1], T[0], -9]))
    assert cache.error() == 0 and torch.equal(cache.page_table[5], cache.page_table[1])
    assert torch.equal(cache.page_table[:5], snap[1][:5])
    invariants(cache, {5: T[1], 1: T[1]})
    want = oracle.forward_direct(x["q"], x["k"], x["v"], x["log_a"], x["lam"])
    got, _ = decode(LL, cache, {k: v[1:2] for k, v in x.items()}, [5], [T[1]], 10)
    check(got[0].cpu(), want[1, T[1]:T[1] + 10])
    # a slot that the row had as its target in the call before, which is not its own now
    now = snapshot(cache)
    LL.loglinear_cache_fork(cache, i32([0, -1]), i32([6, 5]), i32([T[0], T[1]]))
    assert cache.error() == 0 and torch.equal(cache.page_table[:6], now[1][:6])
    assert same([t[5] for t in now[3:]], [t[5] for t in snapshot(cache)[3:]])
    invariants(cache, {6: T[0], 5: T[1] + 10})


def test_a_table_entry_that_is_no_page_counts_for_none(LL):
    """Entries below -1 and past the pool in a table that was overwritten: whoever holds the other
    pages keeps them."""
    cache, x, T = filled(LL)
    for call in (lambda: LL.loglinear_cache_free(cache, i32([2])),
                 lambda: LL.loglinear_cache_reserve(cache, i32([2]), i32([383]))):
        cache.page_table[2] = i32([-2, 10 ** 6, -3, -4])       # (383: block 5 is live and folds into page 1)
        count = cache.refcount.clone()
        call()
        taken = cache.page_table[2][cache.page_table[2] >= 0].tolist()
        taken = [e for e in taken if e < len(count)]
        assert all(count[e] == 0 for e in taken) and len(taken) <= 1
        count[taken] = 1
        assert torch.equal(cache.refcount, count) and cache.error() == 0
    want = oracle.forward_direct(x["q"], x["k"], x["v"], x["log_a"], x["lam"])
    got, _ = decode(LL, cache, {k: v[:2] for k, v in x.items()}, [0, 1], T[:2], 70)
    check(got[0].cpu(), want[0, T[0]:T[0] + 70])
    check(got[1].cpu(), want[1, T[1]:T[1] + 70])


@pytest.mark.parametrize("rows", [1, 160])
@pytest.mark.parametrize("what", ["v", "k", "new v", "new k", "nan"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_fold_of_infinities(LL, dtype, what, rows):
    """An infinite key or value: the page has its infinities where sum_s e k_s v_s has them, NaN
    where that has, and the other elements whole."""
    H, dk, dv, M = 1, 32, 16, 2
    g = torch.Generator().manual_seed(7)
    sign = lambda *s: (0.5 + torch.rand(*s, generator=g)) * (torch.randint(0, 2, s, generator=g) * 2 - 1)  # noqa: E731
    k, v = (sign(1, 64, H, d).to(DT[dtype]) for d in (dk, dv))   # no zeros but one column of values
    v[..., 12] = 0.0
    la = -0.1 * torch.rand(1, 64, H, generator=g)
    at = 63 if "new" in what else 21
    if "v" in what:
        v[0, at, 0, 3], v[0, at, 0, 9] = float("inf"), -float("inf")
    elif "k" in what:
        k[0, at, 0, 5], k[0, at, 0, 30] = float("inf"), -float("inf")
    else:
        k[0, at, 0, 5] = float("nan")
    w = np.exp(to64(la[0, :, 0]).sum() - np.cumsum(to64(la[0, :, 0])))
    with np.errstate(invalid="ignore"):
        want = sum(w[s] * np.outer(to64(k[0, s, 0]), to64(v[0, s, 0])) for s in range(64))
    cache = poison(LL.LogLinearCache.empty(rows, rows, H, dk, dv, M, dtype=DT[dtype]))
    slots = torch.arange(rows, dtype=torch.int32).cuda()
    rep = lambda t: t.expand(rows, *t.shape[1:]).contiguous().cuda()  # noqa: E731
    for t in (slice(0, 63), slice(63, 64)):
        if t.start == 0:
            S = torch.zeros(rows, H, M + 7, dk, dv).cuda()
            LL.loglinear_cache_load(cache, slots, 63, S, rep(k[:, t]), rep(v[:, t]), rep(la[:, t]))
        else:
            p = torch.full_like(slots, 63)
            LL.loglinear_cache_reserve(cache, slots, p)
            lam = torch.ones(rows, H, M + 7).cuda()
            LL.loglinear_cache_step(cache, slots, p, rep(k[:, 63]), rep(k[:, 63]), rep(v[:, 63]), rep(la[:, 63]), lam)
    assert cache.error() == 0
    pages = cache.pages[cache.page_table[:, 0].long()][:, 0].cpu()
    for page in pages[:: max(1, rows // 4)]:
        got = to64(page)
        fin = np.isfinite(want)
        assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~fin], want[~fin], equal_nan=True)
        assert np.all(got[want == 0] == 0) and np.sum(want == 0) >= dk - 2
        check(torch.from_numpy(got[fin]).float(), want[fin])


def test_the_error_word_of_calls_on_another_stream(LL):
    """Read and cleared on the stream that the calls went to, behind them."""
    cache, x, T = filled(LL)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s = i32([99])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)                          # about 10 ms
    LL.loglinear_cache_free(cache, s, stream=side)
    assert cache.error(stream=side) == LL.CACHE_ERR_SLOT
    assert cache.error() == 0 and cache.error(stream=side) == 0
