"""Cases of speculative decoding over the paged decode cache: inputs, plain forms and 64-bit values.

A round of it takes, per sequence, a tree of N drafted tokens whose node 0 is the pending token
(sampled last, not yet in the cache): the tree's attention over the cache, which writes nothing;
the verification of the drafts against the target's probabilities from given random numbers,
which gives the accepted path and the next pending token; and the appending of that path.

The cache keeps, per slot, the raw tokens of the current block of 64 positions, and one fp32 page
[H, d_k, d_v] for every set bit i of (positions >> 6), the state of 2^i blocks; a page's decay since
it was written is one number per head.

`own` selects between the plain forms here (elementary torch operations) and the framework.
"""
import math

import torch

own = False
W = 64        # positions a cache block holds
LOGW = 6
NEG = -1
OUT = -2      # the parent of a node that is left out


# ---------------------------------------------------------------------------- cases

def listed():
    wide = dict(H=16, Hqk=16, dk=128, dv=128, dtype="bf16")
    return [
        # one sequence, a small tree: latency
        dict(name="tree_one", kind="tree", B=1, N=8, pad=0, lo=12345, hi=12345, shape="wide", decay=True, **wide),
        # a server's batch: every sequence at its own position, trees of up to 32 nodes, idle rows
        dict(name="tree_batch", kind="tree", B=64, N=32, pad=3, lo=0, hi=16383, shape="wide", decay=True, **wide),
        # long contexts, one q/k head shared by 48 value heads, trees of 64 nodes
        dict(name="tree_shared", kind="tree", B=24, N=64, pad=0, lo=4096, hi=131071, shape="wide", decay=True, H=48, Hqk=1, dk=128, dv=64, dtype="bf16"),
        # fp32, odd sizes, chains of drafts
        dict(name="tree_f32_chain", kind="tree", B=9, N=5, pad=1, lo=200, hi=5000, shape="chain", decay=True, H=6, Hqk=3, dk=96, dv=36, dtype="f32"),
        # one sequence, drafts given by rank (a tree of a draft model's likeliest tokens)
        dict(name="verify_one", kind="verify", B=1, N=8, pad=0, V=32768, shape="wide", drawn=False, dtype="f32"),
        # a batch of such trees, idle rows, a large vocabulary
        dict(name="verify_batch", kind="verify", B=64, N=32, pad=3, V=131072, shape="wide", drawn=False, dtype="f32"),
        # chains of drafts drawn from the draft model: its probabilities are read too
        dict(name="verify_drawn_chain", kind="verify", B=128, N=6, pad=0, V=131072, shape="chain", drawn=True, dtype="f32"),
        # trees of drawn drafts in bf16, odd vocabulary: rejections redraw among the siblings
        dict(name="verify_drawn_tree", kind="verify", B=32, N=24, pad=0, V=50021, shape="wide", drawn=True, dtype="bf16"),
        # one sequence's accepted path
        dict(name="accept_one", kind="accept", B=1, N=8, D=8, pad=0, lo=12345, hi=12345, cross=False, **wide),
        # a server's batch: some rows reach their block's end
        dict(name="accept_batch", kind="accept", B=128, N=32, D=8, pad=3, lo=0, hi=16383, cross=False, **wide),
        # every row crosses its block's end, one k head shared
        dict(name="accept_cross", kind="accept", B=32, N=16, D=6, pad=0, lo=4096, hi=65535, cross=True, H=48, Hqk=1, dk=128, dv=64, dtype="bf16"),
        # the whole round for a batch
        dict(name="round", kind="round", B=32, N=16, pad=0, lo=100, hi=16383, shape="wide", decay=True, V=65536, drawn=True, pdtype="f32", **wide),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["tree", "tree", "tree", "verify", "verify", "accept", "accept", "round"])
    shape = rng.choice(["wide", "wide", "chain"])
    if kind == "verify":
        N, V = _log(rng, 1, 64), _log(rng, 50, 131072)
        B = _log(rng, 1, max(1, min(128, (1 << 27) // (N * V))))
        return dict(kind=kind, B=B, N=N, pad=rng.randrange(0, max(1, min(4, B))), V=V, shape=shape, drawn=rng.random() < 0.6, dtype=rng.choice(["f32", "f32", "bf16"]))
    heads = rng.choice([(16, 16), (8, 8), (8, 2), (6, 3), (24, 1), (3, 3), (1, 1)])
    dims = rng.choice([(128, 128), (128, 64), (64, 64), (96, 36), (33, 20), (16, 8)])
    c = dict(H=heads[0], Hqk=heads[1], dk=dims[0], dv=dims[1], dtype=rng.choice(["bf16", "bf16", "f32"]))
    lo = _log(rng, 1, 4096) - 1
    hi = lo + _log(rng, 1, 28000)
    B = _log(rng, 1, 64)
    pad = rng.randrange(0, max(1, min(4, B)))
    if kind == "tree":
        return dict(kind=kind, B=B, N=_log(rng, 1, 64), pad=pad, lo=lo, hi=hi, shape=shape, decay=rng.random() < 0.8, **c)
    if kind == "accept":
        N = _log(rng, 1, 64)
        return dict(kind=kind, B=B, N=N, D=rng.randrange(1, min(N, 16) + 1), pad=pad, lo=lo, hi=hi, cross=rng.random() < 0.4, **c)
    N, V = _log(rng, 1, 32), _log(rng, 50, 65536)
    B = min(B, max(1, (1 << 26) // (N * V)))
    return dict(kind=kind, B=B, N=N, pad=0, lo=lo, hi=hi, shape=shape, decay=True, V=V, drawn=rng.random() < 0.6, pdtype=rng.choice(["f32", "bf16"]), **c)


def _dt(name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _spread(i):
    return (0.37 + 0.6180339887498949 * i) % 1.0


def _positions(c):
    """B positions spread over [lo, hi], the same for every seed; `cross`: at most D short of a block's end."""
    pos = [c["lo"] + int(_spread(i) * (c["hi"] - c["lo"] + 1)) for i in range(c["B"])]
    if c.get("cross"):
        pos = [(p | (W - 1)) + 1 - min(c["D"], 1 + i % 4) for i, p in enumerate(pos)]
    return pos


def _parents(c):
    """Each row's tree, the same for every seed: rows differ, and all but the chains and the smallest have some nodes left out."""
    rows = []
    for r in range(c["B"]):
        N = c["N"]
        live = N if c["shape"] == "chain" else max(1, N - int(_spread(r) * N / 4))
        row = [NEG]
        for i in range(1, N):
            row.append(OUT if i >= live else i - 1 if c["shape"] == "chain" else int(_spread(7 * i + 13 * r) * i))
        rows.append([OUT] * N if c["kind"] in ("verify", "round") and r >= c["B"] - c["pad"] else row)
    return rows


def _counts(c):
    """Length of each row's path."""
    return [max(1 + i % 4, 1 + int(_spread(3 * i) * c["D"])) if c.get("cross") else 1 + int(_spread(3 * i) * c["D"]) for i in range(c["B"])]


def _paths(c):
    D, step = c["D"], max(1, c["N"] // c["D"])
    return [[d * step + r % step if d < min(n, D) else NEG for d in range(D)] for r, n in enumerate(_counts(c))]


def _levels(top):
    """Page levels of a cache whose sequences reach position `top`."""
    return max(1, (top >> LOGW).bit_length() + 1)


# ---------------------------------------------------------------------------- inputs

def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    s = dict(c)
    if c["kind"] in ("tree", "verify", "round"):
        s["parents"] = torch.tensor(_parents(c), dtype=torch.int32, device="cuda")
    if c["kind"] != "verify":
        _prepare_cache(c, s, g, rn)
    if c["kind"] in ("verify", "round"):
        _prepare_drafts(c, s, g, rn)
    return s


def _prepare_cache(c, s, g, rn):
    H, Hqk, dk, dv, n, N, dt = c["H"], c["Hqk"], c["dk"], c["dv"], c["B"], c["N"], _dt(c["dtype"])
    pos = _positions(c)
    M = _levels(max(pos) + W)
    S = n + 2
    held = [[i for i in range(M) if (p >> LOGW) >> i & 1] for p in pos]
    P = sum(len(x) for x in held) + n + 3        # room for a fold of every row
    cache = dict(
        pages=rn(P, H, dk, dv).mul_(0.3), page_table=torch.full((S, M), NEG, dtype=torch.int32, device="cuda"),
        refcount=torch.zeros(P, dtype=torch.int32, device="cuda"),
        win_k=(rn(S, Hqk, W, dk) / math.sqrt(dk)).to(dt), win_v=rn(S, H, W, dv).to(dt),
        win_log_a=-0.1 * torch.nn.functional.softplus(rn(S, H, W)),
        page_log=-3.0 * torch.rand(S, 2, M, H, generator=g, device="cuda"),
        page_from=torch.zeros(S, 2, dtype=torch.int32, device="cuda"))
    s["cache"], s["M"], s["L"] = cache, M, LOGW + 1 + M
    slots = torch.randperm(S, generator=g, device="cuda")[:n]
    at = torch.randperm(P, generator=g, device="cuda")     # every sequence's pages, anywhere in the pool
    rows = [i for i, x in enumerate(held) for _ in x]
    if rows:
        lv = torch.tensor([m for x in held for m in x], device="cuda")
        cache["page_table"][slots[torch.tensor(rows, device="cuda")], lv] = at[:len(rows)].to(torch.int32)
        cache["refcount"][at[:len(rows)]] = 1
    s["slots"] = slots.to(torch.int32)
    if c["pad"]:
        s["slots"][n - c["pad"]:] = NEG
    s["pos"] = torch.tensor(pos, dtype=torch.int32, device="cuda")
    s["q"], s["k"] = (rn(n, N, Hqk, dk) / math.sqrt(dk)).to(dt), (rn(n, N, Hqk, dk) / math.sqrt(dk)).to(dt)
    s["v"] = rn(n, N, H, dv).to(dt)
    s["log_a"] = -0.1 * torch.nn.functional.softplus(rn(n, N, H)) if c.get("decay", True) else None
    s["lam"] = torch.nn.functional.softplus(rn(n, N, H, s["L"]))
    s["out"] = torch.zeros(n, N, H, dv, dtype=dt, device="cuda")
    s["new_pos"] = torch.zeros(n, dtype=torch.int32, device="cuda")
    if c["kind"] == "accept":
        s["path"] = torch.tensor(_paths(c), dtype=torch.int32, device="cuda")


def _prepare_drafts(c, s, g, rn):
    """Probabilities of a target and of a draft model that resembles it, and drafts: each node's
    children drawn from the draft's row (`drawn`), or its likeliest tokens."""
    n, N, V, dt = c["B"], c["N"], c["V"], _dt(c.get("pdtype", c["dtype"]))
    logits = rn(n, N, V).mul_(2.5)
    draft = torch.softmax(logits, -1).to(dt)
    s["probs"] = torch.softmax(logits.add_(rn(n, N, V).mul_(0.7)), -1).to(dt)
    del logits
    s["u"] = torch.rand(n, N, generator=g, device="cuda")
    up = s["parents"].clamp(min=0).long()
    row = torch.arange(n, device="cuda")[:, None]
    if c["drawn"]:
        x = torch.rand(n, N, generator=g, device="cuda", dtype=torch.float64)
        tokens = torch.empty(n, N, dtype=torch.int64, device="cuda")
        for i in range(N):      # node i's token from its parent's row, by the sums of it
            cum = draft[row[:, 0], up[:, i]].double().cumsum(-1)
            tokens[:, i] = (cum <= x[:, i:i + 1] * cum[:, -1:]).sum(-1).clamp(max=V - 1)
        s["draft"] = draft
    else:
        same = (up[:, :, None] == up[:, None]) & (s["parents"][:, None] >= 0)
        rank = torch.tril(same, -1).sum(-1)              # among its siblings
        most = min(V, int(rank.max()) + 1)
        best = torch.stack([draft[r].float().topk(most, -1).indices for r in range(n)])
        tokens = best[row, up, rank.clamp(max=most - 1)]
        s["draft"] = None
    s["tokens"] = tokens.to(torch.int32)


# ---------------------------------------------------------------------------- the pass

def run(s):
    kind = s["kind"]
    if own:
        import log_linear_attention_fwd_gb300 as LL
        c = s.get("cache")
        h = s.get("handle")
        if h is None and c is not None:
            h = s["handle"] = LL.LogLinearCache(**c)
        out = {}
        if kind in ("tree", "round"):
            LL.loglinear_cache_tree(h, s["slots"], s["pos"], s["parents"], s["q"], s["k"], s["v"], s["log_a"], s["lam"], out=s["out"])
            out["out"] = s["out"]
        path = s.get("path")
        if kind in ("verify", "round"):
            path, count, token = LL.loglinear_tree_verify(s["parents"], s["tokens"], s["probs"], s["u"], draft=s["draft"])
            out.update(path=path, count=count, token=token)
        if kind in ("accept", "round"):
            LL.loglinear_cache_accept(h, s["slots"], s["pos"], path, s["k"], s["v"], s["log_a"], new_pos=s["new_pos"])
            out.update(new_pos=s["new_pos"], **c)
        return out
    out = {}
    if kind in ("tree", "round"):
        _tree(s["cache"], s)
        out["out"] = s["out"]
    path = s.get("path")
    if kind in ("verify", "round"):
        path, count, token = _verify(s["parents"], s["tokens"].long(), s["probs"], s["u"], s["draft"])
        out.update(path=path, count=count, token=token)
    if kind in ("accept", "round"):
        _accept(s["cache"], s, path)
        out.update(new_pos=s["new_pos"], **s["cache"])
    return out


# ---------------------------------------------------------------------------- plain forms

def _bit_length(x):
    return torch.frexp(x.double())[1].long()


def _ctz(x):
    return _bit_length(x & -x) - 1


def _release(c, at, keep):
    """Slots `at` give up their pages but those whose bit is set in `keep`."""
    M = c["page_table"].shape[1]
    row = c["page_table"][at]
    drop = (row >= 0) & ((keep[:, None] >> torch.arange(M, device="cuda")) & 1 == 0)
    c["refcount"].index_add_(0, row[drop].long(), torch.full((int(drop.sum()),), -1, dtype=torch.int32, device="cuda"))
    c["page_table"][at] = torch.where(drop, torch.full_like(row, NEG), row)


def _take(c, at, want):
    """The lowest free pages for the (slot, level) pairs that `want` marks, in order."""
    free = (c["refcount"] == 0).nonzero()[:, 0][:int(want.sum())]
    row = c["page_table"][at]
    row[want] = free.to(torch.int32)
    c["refcount"][free] = 1
    c["page_table"][at] = row


def _decays(c, at, t):
    """log decay from each window token, and from the pages' reference, up to position t - 1."""
    j, r = t >> LOGW, t & (W - 1)
    i = torch.arange(W, device="cuda")
    la = torch.where((i < r[:, None])[:, None], c["win_log_a"][at].double(), torch.zeros((), dtype=torch.float64, device="cuda"))
    back = la.flip(-1).cumsum(-1).flip(-1)                       # sum over u >= s
    after = torch.cat([back[..., 1:], torch.zeros_like(back[..., :1])], -1)
    start = c["page_from"][at, j & 1].long()
    pad = torch.cat([back, torch.zeros_like(back[..., :1])], -1)
    since = pad.gather(-1, start[:, None, None].expand(-1, la.shape[1], 1))[..., 0]
    return after.float(), (c["page_log"][at, j & 1].double() + since[:, None]).float()  # [n, H, W], [n, M, H]


def _tree(c, s):
    on = (s["slots"] >= 0).nonzero()[:, 0]
    at, pos, up = s["slots"][on].long(), s["pos"][on].long(), s["parents"][on].long()
    n, N, H, M = len(on), up.shape[1], s["v"].shape[2], s["M"]
    G = H // s["k"].shape[2]
    q, k = (s[x][on].float().repeat_interleave(G, 2).transpose(1, 2) for x in ("q", "k"))    # [n, H, N, dk]
    v, lam = s["v"][on].float().transpose(1, 2), s["lam"][on].transpose(1, 2)                  # [n, H, N, L]
    la = s["log_a"][on].transpose(1, 2) if s["log_a"] is not None else torch.zeros(n, H, N, device="cuda")
    # each node's depth, ancestors (and itself), log decay behind each of them and behind the context
    row = torch.arange(n, device="cuda")
    depth = torch.zeros(n, N, dtype=torch.int64, device="cuda")
    anc = torch.zeros(n, N, N, dtype=torch.bool, device="cuda")
    back = torch.zeros(n, H, N, N, device="cuda")
    first = torch.zeros(n, H, N, device="cuda")
    for i in range(N):
        p = up[:, i].clamp(min=0)
        child = up[:, i] >= 0
        depth[:, i] = torch.where(child, depth[row, p] + 1, torch.zeros_like(p))
        anc[:, i] = anc[row, p] & child[:, None]
        back[:, :, i] = torch.where(anc[:, None, i], back[row, :, p] + la[:, :, i, None], torch.zeros((), device="cuda"))
        first[:, :, i] = torch.where(child[:, None], first[row, :, p], torch.zeros((), device="cuda")) + la[:, :, i]
        anc[:, i, i] = up[:, i] >= NEG
    t = pos[:, None] + depth                                                                     # [n, N]
    j, r = pos >> LOGW, pos & (W - 1)
    tok, page = _decays(c, at, pos)
    # the block's tokens
    i = torch.arange(W, device="cuda")
    inside = i < r[:, None]
    wk, wv = c["win_k"][at].float().repeat_interleave(G, 1), c["win_v"][at].float()
    wv = torch.where(inside[:, None, :, None], wv, torch.zeros((), device="cuda"))
    lev = _bit_length(t[:, :, None] ^ ((j << LOGW)[:, None, None] + i))
    p = lam.gather(3, lev[:, None].expand(-1, H, -1, -1)) * torch.exp(tok[:, :, None] + first[..., None]) * torch.matmul(q, wk.transpose(2, 3))
    o = torch.matmul(torch.where(inside[:, None, None], p, torch.zeros((), device="cuda")), wv)
    # the nodes above, and itself
    lev = _bit_length(t[:, :, None] ^ t[:, None])
    p = lam.gather(3, lev.clamp(max=lam.shape[3] - 1)[:, None].expand(-1, H, -1, -1)) * torch.exp(back) * torch.matmul(q, k.transpose(2, 3))
    o = o + torch.matmul(torch.where(anc[:, None], p, torch.zeros((), device="cuda")), torch.where((up >= NEG)[:, None, :, None], v, torch.zeros((), device="cuda")))
    # the pages
    later = (t >> LOGW) > j[:, None]
    for m in range(M):
        live = (j >> m & 1 == 1).nonzero()[:, 0]
        if len(live) == 0:
            continue
        lev = LOGW + 1 + torch.where(later[live], _ctz(j[live] + 1)[:, None].clamp(min=m), torch.full_like(t[live], m))
        w = lam[live].gather(3, lev[:, None, :, None].expand(-1, H, -1, 1)) * torch.exp(page[live, m][:, :, None] + first[live])[..., None]
        o[live] += w * torch.matmul(q[live], c["pages"][c["page_table"][at[live], m].long()])
    o = o.transpose(1, 2).to(s["out"].dtype)
    s["out"][on] = torch.where((up >= NEG)[:, :, None, None], o, s["out"][on])


def _verify(parents, tokens, probs, u, draft):
    """The walk from node 0: parents come before their children, so one pass over the nodes in
    order meets a node's children after it, in their order."""
    n, N, V = probs.shape
    row = torch.arange(n, device="cuda")
    on = parents[:, 0] == NEG
    cur = torch.zeros(n, dtype=torch.int64, device="cuda")
    path = torch.full((n, N), NEG, dtype=torch.int64, device="cuda")
    path[:, 0] = torch.where(on, cur, path[:, 0])
    count = on.long()
    S = torch.zeros(n, dtype=torch.float64, device="cuda")       # sum of the masses so far: what q has been taken off
    Z = torch.ones(n, dtype=torch.float64, device="cuda")        # mass that is left
    gone = torch.full((n, N), NEG, dtype=torch.int64, device="cuda")  # rejected tokens (drafts that were given)
    for i in range(1, N):
        child = on & (parents[:, i] == cur)
        x = tokens[:, i]
        px, un = probs[row, cur, x].double(), u[:, i].double()
        if draft is None:
            left = torch.where((gone == x[:, None]).any(1), torch.zeros_like(px), px)
            ok = child & (un * Z < left)
            no = child & ~ok
            Z = torch.where(no, (Z - left).clamp(min=0), Z)
            gone[:, i] = torch.where(no, x, gone[:, i])
        else:
            qx = draft[row, cur, x].double()
            ok = child & (un * Z * qx < (px - S * qx).clamp(min=0))
            no = (child & ~ok).nonzero()[:, 0]
            S[no] += Z[no]
            Z[no] = (probs[no, cur[no]].double() - S[no, None] * draft[no, cur[no]].double()).clamp(min=0).sum(-1)
        cur = torch.where(ok, torch.full_like(cur, i), cur)
        path[row, count.clamp(max=N - 1)] = torch.where(ok, cur, path[row, count.clamp(max=N - 1)])
        count = count + ok
        S, Z = torch.where(ok, torch.zeros_like(S), S), torch.where(ok, torch.ones_like(Z), Z)
        gone = torch.where(ok[:, None], torch.full_like(gone, NEG), gone)
    full = probs[row, cur].double()
    if draft is None:
        mass = torch.cat([full, torch.zeros_like(full[:, :1])], 1)
        mass = mass.scatter(1, torch.where(gone >= 0, gone, torch.full_like(gone, V)), 0.0)[:, :V]
    else:
        mass = (full - S[:, None] * draft[row, cur].double()).clamp(min=0)
    cum = torch.where((mass > 0).any(1, keepdim=True), mass, full).cumsum(-1)
    token = (cum <= u[:, :1].double() * cum[:, -1:]).sum(-1)
    token = torch.where(on & (token < V), token, torch.full_like(token, NEG))
    return path.to(torch.int32), count.to(torch.int32), token.to(torch.int32)


def _accept(c, s, path):
    """The path's nodes appended as single steps would, token after token."""
    count = (path >= 0).long().cumprod(1).sum(1)
    on = (s["slots"] >= 0).nonzero()[:, 0]
    at, pos, count, path = s["slots"][on].long(), s["pos"][on].long(), count[on], path[on].long()
    j = pos >> LOGW
    to = _ctz(j + 1)
    cross = (pos & (W - 1)) + count >= W                        # a block ends
    _release(c, at, j | torch.where(cross, 1 << to, torch.zeros_like(to)))
    m = torch.arange(c["page_table"].shape[1], device="cuda")
    _take(c, at, cross[:, None] & (m == to[:, None]) & (c["page_table"][at] < 0))
    s["new_pos"][on] = (pos + count).to(torch.int32)
    for d in range(path.shape[1]):
        go = (count > d).nonzero()[:, 0]
        if len(go) == 0:
            break
        b, node = on[go], path[go, d]
        la = s["log_a"][b, node] if s["log_a"] is not None else torch.zeros(len(go), s["v"].shape[2], device="cuda")
        _append(c, at[go], pos[go] + d, s["k"][b, node], s["v"][b, node], la)


def _append(c, at, t, k, v, la):
    H, G, M = v.shape[1], v.shape[1] // k.shape[1], c["page_table"].shape[1]
    r = t & (W - 1)
    c["win_k"][at, :, r], c["win_v"][at, :, r], c["win_log_a"][at, :, r] = k, v, la
    f = (r == W - 1).nonzero()[:, 0]                              # blocks that end here
    if len(f) == 0:
        return
    at, t, la = at[f], t[f], la[f]
    j = t >> LOGW
    to = _ctz(j + 1)
    tok, page = _decays(c, at, t)
    e, log = torch.exp(tok + la[..., None]), page + la[:, None]
    e[..., W - 1] = 1.0
    wk, wv = c["win_k"][at].float().repeat_interleave(G, 1), c["win_v"][at].float()
    new = torch.matmul((e[..., None] * wk).transpose(2, 3), wv)
    m = torch.arange(M, device="cuda")
    for i in range(M):
        low = ((j >> i & 1 == 1) & (i < to)).nonzero()[:, 0]
        if len(low):
            new[low] += torch.exp(log[low, i])[..., None, None] * c["pages"][c["page_table"][at[low], i].long()]
    c["pages"][c["page_table"][at, to].long()] = new
    after = (j + 1)[:, None] >> m & 1 == 1
    log = torch.where((m == to[:, None])[..., None], torch.zeros_like(log), log)
    c["page_log"][at, (j + 1) & 1] = torch.where(after[..., None], log, c["page_log"][at, (j + 1) & 1])
    c["page_from"][at, (j + 1) & 1] = 0


# ---------------------------------------------------------------------------- what a pass needs

def work(c):
    b = f = 0
    size = {"f32": 4, "bf16": 2}
    n = c["B"] - c["pad"]
    if c["kind"] in ("verify", "round"):
        # the last node's row (the draft's too where drawn: a chain or tree ends in a rejection or at a leaf), and two values per node
        e = size[c.get("pdtype", c["dtype"])]
        per = 2 if c["drawn"] else 1
        b += n * (c["V"] * e * per + c["N"] * (2 * e + 16))
        f += 4 * n * c["V"] * per
    if c["kind"] == "verify":
        return {"bytes": b, "flops": f}
    e, H, Hqk, dk, dv, N = size[c["dtype"]], c["H"], c["Hqk"], c["dk"], c["dv"], c["N"]
    page, token = 4 * H * dk * dv, e * (Hqk * dk + H * dv) + 4 * H
    pos = _positions(c)[:n]
    if c["kind"] in ("tree", "round"):
        for p, up in zip(pos, _parents(c)):
            j, r, live, above = p >> LOGW, p & (W - 1), 0, []
            for u in up:
                above.append(0 if u == OUT else 1 if u < 0 else 1 + above[u])
                live += u != OUT
            levels = r.bit_length() + bin(j).count("1") + 1
            b += page * bin(j).count("1") + token * (r + live) + live * (e * (Hqk * dk + H * dv) + 4 * H * levels)
            f += 2 * H * dk * dv * live * bin(j).count("1") + 2 * H * (dk + dv) * (live * r + sum(above))
    if c["kind"] == "accept":
        for p, m in zip(pos, _counts(c)):
            m = min(m, c["D"])
            b += 2 * token * m
            if (p & (W - 1)) + m >= W:
                j = p >> LOGW
                to = ((j + 1) & -(j + 1)).bit_length() - 1
                b += page * (1 + to) + token * (p & (W - 1))
                f += 2 * H * dk * dv * (W + to)
    if c["kind"] == "round":
        b += sum(4 * token for _ in pos)          # about two tokens stay, and are written
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------------------- 64 bits

def exact(c, seed):
    """run()'s values in 64 bits: the attention node by node, the walk and the folds row by row."""
    s = prepare(c, seed)
    out = {}
    if c["kind"] in ("tree", "round"):
        out["out"] = _exact_tree(c, s)
    path = s["path"].tolist() if c["kind"] == "accept" else None
    if c["kind"] in ("verify", "round"):
        path, count, token = _exact_verify(c, s)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        out.update(path=i32(path), count=i32(count), token=i32(token))
    if c["kind"] in ("accept", "round"):
        out.update(_exact_accept(c, s, path))
    return out


def _since(cache, slot, r, j):
    """Log decays in the block: of each token up to the context's last one, and of its pages."""
    la = cache["win_log_a"][slot, :, :r].double()
    return la, la[:, int(cache["page_from"][slot, j & 1]):].sum(1)


def _exact_tree(c, s):
    cache, G = s["cache"], c["H"] // c["Hqk"]
    out = s["out"].double()
    for row, (slot, pos, up) in enumerate(zip(s["slots"].tolist(), s["pos"].tolist(), s["parents"].tolist())):
        if slot < 0:
            continue
        j, r = pos // W, pos % W
        las, since = _since(cache, slot, r, j)
        ks = cache["win_k"][slot, :, :r].double().repeat_interleave(G, 0)
        vs = cache["win_v"][slot, :, :r].double()
        bits = [m for m in range(s["M"]) if j >> m & 1]
        P = torch.stack([cache["pages"][int(cache["page_table"][slot, m])].double() for m in bits]) if bits else None
        log = torch.stack([cache["page_log"][slot, j & 1, m].double() + since for m in bits]) if bits else None   # [P, H]
        q = s["q"][row].double().repeat_interleave(G, 1)
        k = s["k"][row].double().repeat_interleave(G, 1)
        v, lam = s["v"][row].double(), s["lam"][row].double()
        la = s["log_a"][row].double() if s["log_a"] is not None else torch.zeros(c["N"], c["H"], dtype=torch.float64, device="cuda")
        held = torch.einsum("nhd,phde->pnhe", q, P) if bits else None
        for i, u in enumerate(up):
            if u < NEG:
                continue
            line = [i]
            while up[line[0]] >= 0:
                line.insert(0, up[line[0]])
            t = pos + len(line) - 1
            where = list(range(j * W, pos)) + list(range(pos, t + 1))
            al = torch.cat([las, la[line].T], 1)
            K = torch.cat([ks, k[line].transpose(0, 1)], 1)
            V = torch.cat([vs, v[line].transpose(0, 1)], 1)
            dec = (al.sum(1, keepdim=True) - al.cumsum(1)).exp()
            lev = torch.tensor([(t ^ x).bit_length() for x in where], device="cuda")
            o = torch.einsum("hs,hse->he", (K * q[i][:, None]).sum(-1) * dec * lam[i][:, lev], V)
            if bits:
                first = la[line].sum(0)
                # page m holds the blocks from ((j >> m) - 1) << m on: all of one level from t's block
                lv = torch.tensor([LOGW + (t // W ^ ((j >> m) - 1 << m)).bit_length() for m in bits], device="cuda")
                o = o + ((log + first).exp()[:, :, None] * lam[i][:, lv].T[:, :, None] * held[:, i]).sum(0)
            out[row, i] = o
    return out


def _exact_verify(c, s):
    paths, counts, tokens = [], [], []
    every = [s[x].tolist() for x in ("parents", "tokens", "u")]
    for row, (up, tok, u) in enumerate(zip(*every)):
        path, cur = [], 0
        if up[0] == NEG:
            path.append(0)
            while True:
                P = s["probs"][row, cur].double()
                left = P.clone()
                mass, nxt = 1.0, None
                Q = s["draft"][row, cur].double() if s["draft"] is not None else None
                for i in range(cur + 1, c["N"]):
                    if up[i] != cur:
                        continue
                    here = float(left[tok[i]])
                    if u[i] * mass * (1.0 if Q is None else float(Q[tok[i]])) < here:
                        nxt = i
                        break
                    if Q is None:
                        left[tok[i]] = 0.0
                        mass = max(mass - here, 0.0)
                    else:
                        left = (left - mass * Q).clamp(min=0)
                        mass = float(left.sum())
                if nxt is None:
                    break
                path.append(nxt)
                cur = nxt
            if float(left.sum()) <= 0:
                left = P
            cum = left.cumsum(0)
            hit = (cum > u[0] * cum[-1]).nonzero()
            tokens.append(int(hit[0]) if len(hit) else NEG)
        else:
            tokens.append(NEG)
        counts.append(len(path))
        paths.append(path + [NEG] * (c["N"] - len(path)))
    return paths, counts, tokens


def _exact_accept(c, s, paths):
    cache, G = s["cache"], c["H"] // c["Hqk"]
    # tables and counts: whole numbers, settled before anything is computed
    rows = [(b, slot, pos, [x for x in path if x >= 0]) for b, (slot, pos, path) in
            enumerate(zip(s["slots"].tolist(), s["pos"].tolist(), paths)) if slot >= 0]
    table, count = cache["page_table"].tolist(), cache["refcount"].tolist()
    ends = []
    for b, slot, pos, path in rows:
        j = pos // W
        to = ((j + 1) & -(j + 1)).bit_length() - 1
        end = pos % W + len(path) >= W
        for m in range(s["M"]):
            if table[slot][m] >= 0 and not (j >> m & 1 or (end and m == to)):
                count[table[slot][m]] -= 1
                table[slot][m] = NEG
        ends.append((j, to, end))
    free = iter([p for p, x in enumerate(count) if x == 0])
    for (b, slot, pos, path), (j, to, end) in zip(rows, ends):
        if end and table[slot][to] < 0:
            table[slot][to] = next(free)
            count[table[slot][to]] = 1
    new = {x: cache[x].double() for x in ("pages", "win_k", "win_v", "win_log_a", "page_log")}
    new["page_from"], new_pos = cache["page_from"].clone(), s["new_pos"].clone()
    pages = cache["pages"]
    for (b, slot, pos, path), (j, to, end) in zip(rows, ends):
        new_pos[b] = pos + len(path)
        k, v = s["k"][b, path].double(), s["v"][b, path].double()             # [d, Hqk, dk], [d, H, dv]
        la = s["log_a"][b, path].double() if s["log_a"] is not None else torch.zeros(len(path), c["H"], dtype=torch.float64, device="cuda")
        r = pos % W
        if end:
            a = W - r                                                             # tokens that end the block
            old, since = _since(cache, slot, r, j)
            al = torch.cat([old, la[:a].T], 1)
            K = torch.cat([cache["win_k"][slot, :, :r].double(), k[:a].transpose(0, 1)], 1).repeat_interleave(G, 0)
            V = torch.cat([cache["win_v"][slot, :, :r].double(), v[:a].transpose(0, 1)], 1)
            dec = (al.sum(1, keepdim=True) - al.cumsum(1)).exp()
            page = torch.einsum("hsd,hse->hde", dec[..., None] * K, V)
            start = int(cache["page_from"][slot, j & 1])
            tail = since + la[:a].sum(0) if start <= r else al[:, start:].sum(1)
            for m in range(s["M"]):
                if j >> m & 1:
                    log = cache["page_log"][slot, j & 1, m].double() + tail
                    if m < to:
                        page = page + log.exp()[:, None, None] * pages[table[slot][m]].double()
                    else:
                        new["page_log"][slot, (j + 1) & 1, m] = log
            new["pages"][table[slot][to]] = page
            new["page_log"][slot, (j + 1) & 1, to] = 0
            new["page_from"][slot, (j + 1) & 1] = 0
        for d in range(len(path)):
            x = (pos + d) % W
            new["win_k"][slot, :, x], new["win_v"][slot, :, x], new["win_log_a"][slot, :, x] = k[d], v[d], la[d]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    new.update(page_table=i32(table), refcount=i32(count), new_pos=new_pos)
    return new
