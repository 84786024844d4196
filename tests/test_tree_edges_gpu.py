"""Speculative decoding on the GPU where it is easily wrong: bf16 outputs, deep decays, infinities, rows that do
not sum to 1, and pages that are shared or overwritten, in both forms of the plan.

Tolerances as in tests/test_tree_gpu.py, by the same helpers; each test states what it adds.
"""
import numpy as np
import pytest
import torch

import oracle
from tests.helpers import TOL_F32, rel_l2, to64
from tests.test_cache_gpu import decode, filled, i32, invariants, snapshot
from tests.test_tree_gpu import TWO_PARTS, attend, contexts, parents_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def LL():
    import log_linear_attention_fwd_gb300 as m
    return m


def live_of(parents):
    return torch.tensor(parents).cuda() != -2


@pytest.mark.parametrize("N", [5, 13, 30, 64])
@pytest.mark.parametrize("H,Hqk,dk,dv,dtype", [(4, 2, 128, 128, "bf16"), (6, 1, 128, 64, "bf16"), (2, 2, 72, 100, "bf16"),
                                               (2, 1, 96, 36, "f32")])
def test_bf16_outputs_are_the_fp32_outputs_rounded(LL, H, Hqk, dk, dv, dtype, N):
    """The outputs' type decides about their last rounding only: equal to the bit."""
    pos = [0, 63, 150, 448, 511, 1000]
    parents = parents_of(len(pos), N, "tree")
    cache, slots, ctx, tree, x = contexts(LL, pos, N, H, Hqk, dk, dv, dtype, True)
    wide, narrow = (attend(LL, cache, slots, pos, parents, x, out_dtype=t) for t in (torch.float32, torch.bfloat16))
    live = live_of(parents)
    assert torch.equal(wide[live].bfloat16(), narrow[live])
    assert cache.error() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_deep_decays_that_decide(LL, dtype):
    """Log decays down to -56 under level weights of up to e^56: the terms that have decayed most are the output.
    A sum of log decays below 64 rounds by 2^-19 (half a step) at each of at most 6 additions, and so
    moves its term by 6 2^-19 beside the tests' other bounds; bf16 outputs round that once."""
    pos, N = [70, 200], 4
    cache, slots, ctx, tree, x = contexts(LL, pos, N, 2, 1, 64, 32, dtype, True)
    chain = [[-1, 0, 1, 2]] * 2
    x["log_a"].fill_(-14.0)
    for i in range(N):
        x["lam"][:, i, :, 3:] *= float(np.exp(14.0 * (i + 1)))
        x["lam"][:, i, :, :3] *= 0.125
    for r, t in enumerate(tree):
        t["log_a"], t["lam"] = x["log_a"][r].cpu(), x["lam"][r].cpu()
    want = np.stack([oracle.tree_attention(c, t, p) for c, t, p in zip(ctx, tree, chain)])
    got = attend(LL, cache, slots, pos, chain, x, out_dtype=torch.float32)
    tol = TOL_F32 + TWO_PARTS + 6 * 2.0 ** -19
    for r in range(2):
        for i in range(N):
            assert rel_l2(got[r, i], want[r, i]) <= tol, (r, i, rel_l2(got[r, i], want[r, i]))
    assert torch.equal(attend(LL, cache, slots, pos, chain, x, out_dtype=torch.bfloat16), got.bfloat16())


@pytest.mark.parametrize("rows", [1, 80])
@pytest.mark.parametrize("N", [5, 16, 20, 40])
def test_fp32_trees_lose_no_more_than_their_parts_leave(LL, N, rows):
    """fp32 tokens and outputs, seven pages of random states and no decay.  A term has at most three factors that are
    taken as parts, which leave 2^-22 of each, and three roundings of 2^-24; signs and amounts are random, so
    that together with the sums' own roundings (2^-24 of what stands there, 2^-24 sqrt(128) over a page's rows if all went
    one way by half) the whole is below 2^-21 of the outputs' norm."""
    H, Hqk, d, M = 2, 1, 128, 9
    pos, L = 64 * 0b101111110 + 37, M + 7
    g = torch.Generator().manual_seed(N)
    rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = {"q": rand(1, N, Hqk, d) / 8, "k": rand(1, N, Hqk, d) / 8, "v": rand(1, N, H, d), "lam": torch.rand(1, N, H, L, generator=g)}
    wk, wv, state = rand(1, 37, Hqk, d) / 8, rand(1, 37, H, d), torch.zeros(1, H, L, d, d)
    live = [m for m in range(M) if pos >> 6 >> m & 1]
    for m in live:
        state[0, :, 7 + m] = rand(H, d, d)
    cache = LL.LogLinearCache.empty(1, 10, H, d, d, M, Hqk=Hqk, dtype=torch.float32)
    LL.loglinear_cache_load(cache, i32([0]), pos, state.cuda(), wk.cuda(), wv.cuda(), None)
    assert len(live) == 7 and cache.error() == 0
    chain = [list(range(-1, N - 1))] * rows
    y = {k: v.cuda().repeat(rows, 1, 1, 1) for k, v in x.items()}
    got = attend(LL, cache, [0] * rows, [pos] * rows, chain, dict(y, log_a=None)).cpu()
    q, lam, S = to64(x["q"][0, :, 0]), to64(x["lam"][0]), to64(state[0])
    keys, vals = to64(torch.cat([wk, x["k"]], 1)[0, :, 0]), to64(torch.cat([wv, x["v"]], 1)[0])
    want = np.zeros((N, H, d))
    for i in range(N):
        t = pos + i
        over = t >> 6 != pos >> 6
        to = ((t >> 6) & -(t >> 6)).bit_length() - 1 if over else 0
        w = np.stack([lam[i, :, oracle.level(t, pos - 37 + s)] * (keys[s] @ q[i]) for s in range(38 + i)])
        want[i] = np.einsum("sh,shd->hd", w, vals[:38 + i])
        for m in live:
            want[i] += lam[i, :, 7 + max(m, to), None] * (q[i] @ S[:, 7 + m])
    for r in range(rows):
        assert rel_l2(got[r], want) <= 2.0 ** -21, rel_l2(got[r], want)
    assert cache.error() == 0


@pytest.mark.parametrize("n,H,Hqk,dk,dv,N", [(1, 1, 1, 32, 16, 5), (1, 2, 1, 128, 128, 30), (2, 2, 2, 96, 36, 64), (40, 4, 2, 33, 20, 9),
                                             (40, 4, 1, 128, 64, 64), (24, 8, 2, 128, 128, 17)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_infinities_in_pages(LL, dtype, n, H, Hqk, dk, dv, N):
    """A page's infinities and NaN: the outputs' column has q's sign of them for each node, NaN where q is 0 there or
    two of them are of both signs; every other output is as without them, to the bit.  (Clusters; CTAs by themselves.)"""
    pos = [70 + 64 * (i % 3) for i in range(n)]
    cache, slots, ctx, tree, x = contexts(LL, pos[:3], N, H, Hqk, dk, dv, dtype, True)
    slots = [slots[i % 3] for i in range(n)]
    x = {k: v[[i % len(v) for i in range(n)]].contiguous() for k, v in x.items()}
    x["q"][:, :, :, 3] = x["q"][:, :, :, 3].abs().clamp(min=0.125) * torch.tensor([1.0, -1.0]).repeat(N)[:N].cuda()[None, :, None]
    x["q"][:, 0, :, 3] = 0.0
    x["q"][:, :, :, dk - 1] = x["q"][:, :, :, dk - 1].abs().clamp(min=0.125)
    parents = parents_of(n, N, "tree")
    live = live_of(parents)
    h, where = H - 1, {int(cache.page_table[s, next(m for m in range(5) if p >> 6 >> m & 1)]) for s, p in zip(slots, pos)}
    for e in where:
        cache.pages[e, h, [3, dk - 1], 1] = 0.0
    zeros = lambda: torch.zeros(n, N, H, dv).cuda()  # noqa: E731
    plain = attend(LL, cache, slots, pos, parents, x, out=zeros())
    inf, nan = float("inf"), float("nan")
    for at, last in ((inf, 0.0), (-inf, 0.0), (nan, 0.0), (inf, inf)):
        for e in where:
            cache.pages[e, h, 3, 1], cache.pages[e, h, dk - 1, 1] = at, last
        got = attend(LL, cache, slots, pos, parents, x, out=zeros())
        want = plain.clone()
        want[:, :, h, 1] = x["q"][:, :, h // (H // Hqk), 3].float() * at + x["q"][:, :, h // (H // Hqk), dk - 1].float() * last
        assert not torch.isfinite(want[:, :, h, 1]).any()
        assert torch.equal(got[live].nan_to_num(5.0), want[live].nan_to_num(5.0)), (at, last)
        assert torch.equal(torch.isnan(got[live]), torch.isnan(want[live]))
    assert cache.error() == 0


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("dtype,odt", [("f32", torch.float32), ("bf16", torch.float32), ("bf16", torch.bfloat16)])
def test_an_infinite_weight_on_an_infinite_value(LL, dtype, odt, value):
    """inf * inf is an infinity of the sum, with the signs' product; what the node's other values and the other
    branches get is as without it."""
    pos, N, H, dk, dv = [70], 6, 1, 32, 16
    cache, slots, ctx, tree, x = contexts(LL, pos, N, H, H, dk, dv, dtype, True)
    for name in ("q", "k"):
        x[name].abs_()
        x[name].clamp_(min=0.125)
    parents = [[-1, 0, 1, 1, 2, 0]]
    plain = attend(LL, cache, slots, pos, parents, x, out_dtype=odt)
    x["v"][0, 2, 0, 9] = value
    x["lam"][0, 4, 0, oracle.level(73, 72)] = float("inf")      # node 4 (t 73) from node 2 (t 72)
    got = attend(LL, cache, slots, pos, parents, x, out_dtype=odt)
    same_value = (lambda a: bool(torch.isnan(a))) if value != value else (lambda a: float(a) == value)
    assert same_value(got[0, 4, 0, 9]) and same_value(got[0, 2, 0, 9])
    rest = [c for c in range(dv) if c != 9]
    assert torch.equal(got[0, 4, 0, rest].float(), torch.sign(x["v"][0, 2, 0, rest].float()) * float("inf"))
    assert torch.equal(got[0, 2, 0, rest], plain[0, 2, 0, rest])
    for i in (0, 1, 3, 5):
        assert torch.equal(got[0, i], plain[0, i])


@pytest.mark.parametrize("rows", [1, 310])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_verify_rows_that_sum_to_more(LL, dtype, rows):
    """Rows of 2^17 ones, with drafts that they have at 0: S grows by 2^17 with each rejection, past 2^19 after four
    of them and past 2^21 after seventeen.  What Q has reached is at 0 from the second one on and stays there: a
    token of it is neither accepted nor drawn.  (One row by a cluster; many by a CTA each.)"""
    some, ones = 1000, 2 ** 17
    V, N = some + ones + 8, 30
    probs, draft = (torch.zeros(rows, N, V, dtype=dtype, device="cuda") for _ in range(2))
    probs[-1, 0, :some + ones] = 1.0
    draft[-1, 0, :some], draft[-1, 0, some + ones:] = 2.0 ** -12, 2.0 ** -10
    parents = torch.full((rows, N), -2, dtype=torch.int32).cuda()          # the other rows are padding
    parents[-1] = i32([-1] + [0] * (N - 1))
    for at in (3, 5, 10, 17, 18, 21, 29):                                   # the child that has a token of Q's
        tokens, u = [V - 1] * N, torch.full((N,), 0.25)
        tokens[at], u[0], u[at] = 5, 0.0, 0.0
        assert oracle.tree_verify(parents[-1].tolist(), tokens, probs[-1].cpu(), u, draft[-1].cpu()) == ([0], some)
        path, count, token = LL.loglinear_tree_verify(parents, i32([tokens] * rows), probs, u.repeat(rows, 1).cuda(), draft=draft)
        assert (path[-1].tolist(), int(count[-1]), int(token[-1])) == ([0] + [-1] * (N - 1), 1, some), at
        assert LL.device_error() == 0


def leftover(LL):
    """Slots 0 and 4 at 188, in block 2, with block 1's page of level 0 left over, which is slot 3's live one
    (at 74) too; block 2 folds to that level."""
    cache, x, _ = filled(LL, n=1, T=(64 + 10,), more=160)
    LL.loglinear_cache_fork(cache, i32([0, 0]), i32([3, 4]), i32([74, 74]))
    one = {k: v[:1] for k, v in x.items()}
    two = {k: torch.cat([v, v]) for k, v in one.items()}
    pos = 74
    while pos < 188:
        _, (pos, _) = decode(LL, cache, two, [0, 4], [pos, pos], 1, reserve=pos in (127,))
    page = int(cache.page_table[0, 0])
    assert page >= 0 and (cache.page_table[[0, 3, 4], 0] == page).all() and cache.refcount[page] == 3 and cache.error() == 0
    return cache, one, two, page, oracle.forward_direct(x["q"], x["k"], x["v"], x["log_a"], x["lam"])


def padded(values, rows, fill=-1):
    """values, then `fill` up to `rows` rows (more than 1024: the plan's other form)."""
    return values + [fill] * (rows - len(values))


@pytest.mark.parametrize("rows", [2, 1100])
def test_an_accepted_fold_never_writes_a_shared_page(LL, rows):
    """A page left over where the fold goes, and shared, is replaced: its other holders keep it."""
    cache, one, two, page, want = leftover(LL)
    held, N = cache.pages[page].clone(), 6
    k, v, la = (torch.zeros(rows, N, *one[n].shape[2:], dtype=one[n].dtype).cuda() for n in ("k", "v", "log_a"))
    for t, n in ((k, "k"), (v, "v"), (la, "log_a")):
        t[:2] = two[n][:, 188:194].cuda()
    new = LL.loglinear_cache_accept(cache, i32(padded([0, 4], rows)), i32(padded([188, 188], rows, 0)),
                                    i32([list(range(N))] * rows), k, v, la, new_pos=i32([-9] * rows))
    assert new.tolist() == padded([194, 194], rows, -9) and cache.error() == 0
    assert torch.equal(cache.pages[page], held) and int(cache.page_table[3, 0]) == page and cache.refcount[page] == 1
    mine = cache.page_table[[0, 4], 0].tolist()
    assert len({page, *mine}) == 3 and cache.refcount[mine].tolist() == [1, 1]
    invariants(cache, {0: 194, 4: 194, 3: 74})
    got, _ = decode(LL, cache, two, [0, 4], [194, 194], 40)
    for r in range(2):
        assert rel_l2(got[r].cpu(), want[0, 194:234]) <= TOL_F32
    got, _ = decode(LL, cache, one, [3], [74], 40)
    assert rel_l2(got[0].cpu(), want[0, 74:114]) <= TOL_F32
    assert cache.error() == 0


def test_reservations_of_both_forms_settle_shared_pages_alike(LL):
    """The same rows in a call of 2 and in one of more than 1024: the same tables and counts, and whole outputs."""
    cache, one, two, page, want = leftover(LL)
    _, (pos, _) = decode(LL, cache, two, [0, 4], [188, 188], 3, reserve=False)
    assert pos == 191
    held, twin = cache.pages[page].clone(), LL.LogLinearCache(*snapshot(cache))
    for c, rows in ((cache, 2), (twin, 1100)):
        LL.loglinear_cache_reserve(c, i32(padded([0, 4], rows)), i32(padded([191, 191], rows, 0)))
        assert c.error() == 0 and torch.equal(c.pages[page], held) and c.refcount[page] == 1
    assert torch.equal(cache.page_table, twin.page_table) and torch.equal(cache.refcount, twin.refcount)
    for c in (cache, twin):
        got, _ = decode(LL, c, two, [0, 4], [191, 191], 1, reserve=False)
        tail, _ = decode(LL, c, two, [0, 4], [192, 192], 40)
        for r in range(2):
            assert rel_l2(torch.cat([got, tail], 1)[r].cpu(), want[0, 191:232]) <= TOL_F32
        invariants(c, {0: 232, 4: 232, 3: 74})
        got, _ = decode(LL, c, one, [3], [74], 40)
        assert rel_l2(got[0].cpu(), want[0, 74:114]) <= TOL_F32
        assert c.error() == 0


@pytest.mark.parametrize("rows", [1, 1100])
@pytest.mark.parametrize("call", ["free", "reserve", "accept"])
def test_overwritten_tables_in_both_forms(LL, call, rows):
    """Entries below -1 and past the pool count for no page: whoever holds the others keeps them."""
    cache, x, T = filled(LL)
    cache.page_table[2] = i32([-2, 10 ** 6, -3, -4])
    count = cache.refcount.clone()
    slots = i32(padded([2], rows))
    if call == "free":
        LL.loglinear_cache_free(cache, slots)
    elif call == "reserve":
        LL.loglinear_cache_reserve(cache, slots, i32(padded([383], rows, 0)))   # block 5 is live and folds into level 1
    else:                                                                        # its path ends block 5, whose page of level 0 is not there
        z = lambda *s: torch.zeros(rows, 2, *s).cuda()  # noqa: E731
        new = LL.loglinear_cache_accept(cache, slots, i32(padded([382], rows, 0)), i32([[0, 1]] * rows), z(2, 16), z(2, 8), None,
                                        new_pos=i32([-9] * rows))
        assert (new == -9).all()
    taken = [e for e in cache.page_table[2].tolist() if 0 <= e < len(count)]
    assert len(taken) == (call != "free") and all(count[e] == 0 for e in taken)
    count[taken] = 1
    assert torch.equal(cache.refcount, count)
    assert cache.error() == (LL.CACHE_ERR_MISSING if call == "accept" else 0)
    want = oracle.forward_direct(x["q"], x["k"], x["v"], x["log_a"], x["lam"])
    got, _ = decode(LL, cache, {k: v[:2] for k, v in x.items()}, [0, 1], T[:2], 70)
    for r in range(2):
        assert rel_l2(got[r].cpu(), want[r, T[r]:T[r] + 70]) <= TOL_F32
