"""Cases of the recurrence and decode-cache operators: inputs, plain forms and 64-bit values.

Two families.  The gated linear recurrence, per channel,

    h_t = a_t h_{t-1} + b_t x_t,  a_t = exp(log_a_t),  b_t = 1, 1 - a_t or sqrt(1 - a_t^2),

over whole (or packed) sequences, its gradients, and its single-token step.  And the paged
decode cache of log-linear attention: per slot, the raw tokens of the current block of 64
positions, and one fp32 page [H, d_k, d_v] for every set bit i of (positions >> 6), the state
of 2^i blocks; a page's decay since it was written is one number per head.  Operators on it: the
decode step (with the page reservation that goes before it), loading a prompt's dense states,
storing dense states, forking, freeing and compacting.

`own` selects between the plain forms here (elementary torch operations) and the framework.
"""
import math

import torch

own = False
W = 64        # positions a cache block holds
LOGW = 6
NEG = -1


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # a training forward at the pretraining length, real gates, Griffin's input scale
        dict(name="glr_fwd_t16384", kind="glr_fwd", B=1, T=16384, D=2048, N=0, dtype="bf16", gate="f32", scale="sqrt", h0=False),
        # packed documents of unequal length in fp32, states carried in and out, odd width
        dict(name="glr_fwd_packed", kind="glr_fwd", B=1, T=9001, D=1000, N=37, dtype="f32", gate="f32", scale="none", h0=True),
        # the gradient of a training step over four sequences
        dict(name="glr_bwd_b4t4096", kind="glr_bwd", B=4, T=4096, D=2048, N=0, dtype="bf16", gate="f32", scale="sqrt", h0=False),
        # the gradient over packed documents, with gradients of the first and last states
        dict(name="glr_bwd_packed", kind="glr_bwd", B=1, T=2500, D=514, N=11, dtype="f32", gate="f32", scale="one_minus", h0=True),
        # one token for each of 128 sequences, states held in slots
        dict(name="glr_step_b128", kind="glr_step", B=128, S=160, D=2048, dtype="bf16", gate="f32", scale="sqrt"),
        # one sequence, one token: latency
        dict(name="cache_step_one", kind="cache_step", B=1, pad=0, lo=12345, hi=12345, H=16, Hqk=16, dk=128, dv=128, dtype="bf16", decay=True),
        # a server's batch: every sequence at its own position, a few rows idle
        dict(name="cache_step_batch", kind="cache_step", B=128, pad=3, lo=0, hi=16383, H=16, Hqk=16, dk=128, dv=128, dtype="bf16", decay=True),
        # long contexts, one q/k head shared by 48 value heads
        dict(name="cache_step_shared", kind="cache_step", B=32, pad=0, lo=4096, hi=131071, H=48, Hqk=1, dk=128, dv=64, dtype="bf16", decay=True),
        # prompts enter the cache from their prefill
        dict(name="cache_load", kind="cache_load", n=32, T=12345, H=16, Hqk=16, dk=128, dv=128, dtype="bf16"),
        # sequences leave it (preemption, moving to another cache)
        dict(name="cache_store", kind="cache_store", n=16, lo=1, hi=16383, H=16, Hqk=16, dk=128, dv=128, dtype="bf16"),
        # four samples from each prompt
        dict(name="cache_fork", kind="cache_fork", n=16, copies=4, lo=100, hi=16383, H=16, Hqk=16, dk=128, dv=128, dtype="bf16"),
        # a batch ends, the pool is compacted, the next batch enters; twice
        dict(name="cache_churn", kind="cache_churn", n=16, T=16383, H=16, Hqk=16, dk=128, dv=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["glr_fwd", "glr_fwd", "glr_bwd", "glr_bwd", "glr_step", "cache_step", "cache_step", "cache_step", "cache_load", "cache_store", "cache_fork", "cache_churn"])
    types = rng.choice([("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
    scale = rng.choice(["none", "one_minus", "sqrt"])
    if kind in ("glr_fwd", "glr_bwd"):
        D, packed = _log(rng, 1, 4096), rng.random() < 0.5
        most = (1 << 24) // D
        if packed:
            T = _log(rng, 1, min(65536, most))
            return dict(kind=kind, B=1, T=T, D=D, N=_log(rng, 1, 64), dtype=types[0], gate=types[1], scale=scale, h0=rng.random() < 0.5)
        B = _log(rng, 1, min(32, most))
        return dict(kind=kind, B=B, T=_log(rng, 1, min(65536, most // B)), D=D, N=0, dtype=types[0], gate=types[1], scale=scale, h0=rng.random() < 0.5)
    if kind == "glr_step":
        B = _log(rng, 1, 512)
        return dict(kind=kind, B=B, S=B + rng.randrange(0, 33), D=_log(rng, 1, 4096), dtype=types[0], gate=types[1], scale=scale)
    heads = rng.choice([(16, 16), (8, 8), (8, 2), (6, 3), (24, 1), (3, 3), (1, 1)])
    dims = rng.choice([(128, 128), (128, 64), (64, 64), (96, 36), (33, 20), (16, 8)])
    c = dict(H=heads[0], Hqk=heads[1], dk=dims[0], dv=dims[1], dtype=types[0])
    lo = _log(rng, 1, 4096) - 1
    hi = lo + _log(rng, 1, 28000)
    if kind == "cache_step":
        B = _log(rng, 1, 128)
        return dict(kind=kind, B=B, pad=rng.randrange(0, max(1, min(4, B))), lo=lo, hi=hi, decay=rng.random() < 0.8, **c)
    if kind == "cache_load":
        return dict(kind=kind, n=_log(rng, 1, 32), T=rng.choice([hi, (hi >> LOGW) << LOGW, hi | 63]), **c)
    if kind == "cache_store":
        return dict(kind=kind, n=_log(rng, 1, 16), lo=lo, hi=hi, **c)
    if kind == "cache_fork":
        return dict(kind=kind, n=_log(rng, 1, 32), copies=rng.randrange(1, 5), lo=lo, hi=hi, **c)
    return dict(kind=kind, n=_log(rng, 1, 16), T=_log(rng, 64, 16384), **c)


def _dt(name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _positions(c, n):
    """n positions spread over [lo, hi], the same for every seed."""
    return [c["lo"] + int(((0.37 + 0.6180339887498949 * i) % 1.0) * (c["hi"] - c["lo"] + 1)) for i in range(n)]


def _cuts(c):
    """Bounds of N packed sequences in [0, T], of unequal length, some empty."""
    N, T = c["N"], c["T"]
    w = [0 if i % 7 == 5 and N > 7 else 1 + (i * i * 31 + 17) % 97 for i in range(N)]
    cu, total, s = [0], sum(w), 0
    for x in w:
        s += x
        cu.append(T * s // total)
    return cu


def _levels(top):
    """Page levels of a cache whose sequences reach position `top`."""
    return max(1, (top >> LOGW).bit_length() + 1)


# ---------------------------------------------------------------------------- inputs

def _gates(g, shape, D, dt):
    base = torch.log(0.9 + 0.099 * torch.rand(D, generator=g, device="cuda"))
    return (8.0 * base * torch.sigmoid(torch.randn(shape, generator=g, device="cuda"))).to(dt)


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    kind, dt = c["kind"], _dt(c["dtype"])
    s = dict(c)
    if kind in ("glr_fwd", "glr_bwd"):
        B, T, D = c["B"], c["T"], c["D"]
        n = c["N"] or B
        s["x"] = rn(B, T, D).to(dt)
        s["log_a"] = _gates(g, (B, T, D), D, _dt(c["gate"]))
        s["h0_"] = rn(n, D) if c["h0"] else None
        s["cu"] = torch.tensor(_cuts(c), dtype=torch.int32, device="cuda") if c["N"] else None
        if kind == "glr_fwd":
            s["state"] = torch.empty(n, D, device="cuda")
        else:
            s["out"] = rn(B, T, D).to(dt)     # what the forward gave: h_t
            s["dout"] = rn(B, T, D).to(dt)
            s["dstate"] = rn(n, D) if c["h0"] else None
        return s
    if kind == "glr_step":
        B, S, D = c["B"], c["S"], c["D"]
        s["x"], s["log_a"] = rn(B, D).to(dt), _gates(g, (B, D), D, _dt(c["gate"]))
        s["state"] = rn(S, D)
        s["slots"] = torch.randperm(S, generator=g, device="cuda")[:B].to(torch.int32)
        return s
    return _prepare_cache(c, s, g, rn, dt)


def _prepare_cache(c, s, g, rn, dt):
    kind, H, Hqk, dk, dv = c["kind"], c["H"], c["Hqk"], c["dk"], c["dv"]
    if kind == "cache_step":
        n, pos = c["B"], _positions(c, c["B"])
        top = c["hi"] + 1
    elif kind in ("cache_store", "cache_fork"):
        n, pos, top = c["n"], _positions(c, c["n"]), c["hi"]
    else:
        n, pos, top = c["n"], [], c["T"]
    S = {"cache_step": n + 2, "cache_load": n, "cache_store": n, "cache_fork": n * (1 + c.get("copies", 0)), "cache_churn": 2 * n}[kind]
    M = _levels(top)
    held = [[i for i in range(M) if (p >> LOGW) >> i & 1] for p in pos]
    if kind in ("cache_load", "cache_churn"):
        P = n * bin(c["T"] >> LOGW).count("1") * (2 if kind == "cache_churn" else 1)
    else:
        P = sum(len(x) for x in held) + sum(p & (W - 1) == W - 1 for p in pos)
    P = max(P, 1) + 3
    cache = dict(
        pages=rn(P, H, dk, dv).mul_(0.3), page_table=torch.full((S, M), NEG, dtype=torch.int32, device="cuda"),
        refcount=torch.zeros(P, dtype=torch.int32, device="cuda"),
        win_k=(rn(S, Hqk, W, dk) / math.sqrt(dk)).to(dt), win_v=rn(S, H, W, dv).to(dt),
        win_log_a=-0.1 * torch.nn.functional.softplus(rn(S, H, W)),
        page_log=-3.0 * torch.rand(S, 2, M, H, generator=g, device="cuda"),
        page_from=torch.zeros(S, 2, dtype=torch.int32, device="cuda"))
    s["cache"], s["M"] = cache, M
    slots = torch.randperm(S, generator=g, device="cuda")
    if pos:  # every sequence's pages, anywhere in the pool
        at = torch.randperm(P, generator=g, device="cuda")
        rows = [i for i, x in enumerate(held) for _ in x]
        if rows:
            lv = torch.tensor([m for x in held for m in x], device="cuda")
            cache["page_table"][slots[:n][torch.tensor(rows, device="cuda")], lv] = at[:len(rows)].to(torch.int32)
            cache["refcount"][at[:len(rows)]] = 1
        s["pos"] = torch.tensor(pos, dtype=torch.int32, device="cuda")
    s["slots"] = slots[:n].to(torch.int32)
    L = LOGW + 1 + M
    s["L"] = L
    if kind == "cache_step":
        if c["pad"]:
            s["slots"][n - c["pad"]:] = NEG
        s["q"], s["k"] = (rn(n, Hqk, dk) / math.sqrt(dk)).to(dt), (rn(n, Hqk, dk) / math.sqrt(dk)).to(dt)
        s["v"] = rn(n, H, dv).to(dt)
        s["log_a"] = -0.1 * torch.nn.functional.softplus(rn(n, H)) if c["decay"] else None
        s["lam"] = torch.nn.functional.softplus(rn(n, H, L))
        s["out"] = torch.zeros(n, H, dv, dtype=dt, device="cuda")
    elif kind == "cache_store":
        s["dense"] = torch.empty(n, H, L, dk, dv, device="cuda")
    elif kind == "cache_fork":
        r = c["copies"]
        s["src"] = s["slots"].repeat_interleave(r)
        s["dst"] = slots[n:].to(torch.int32).contiguous()
        s["pos"] = s["pos"].repeat_interleave(r)
    else:
        for name, sl in (("a", slots[:n]), ("b", slots[n:])):
            if name == "b" and kind == "cache_load":
                break
            s[name] = dict(slots=sl.to(torch.int32).contiguous(), state=rn(n, H, L, dk, dv).mul_(0.3),
                           k=(rn(n, W, Hqk, dk) / math.sqrt(dk)).to(dt), v=rn(n, W, H, dv).to(dt),
                           log_a=-0.1 * torch.nn.functional.softplus(rn(n, W, H)))
        if kind == "cache_churn":
            _load(cache, s["a"], c["T"])
            _load(cache, s["b"], c["T"])
    return s


# ---------------------------------------------------------------------------- the pass

def run(s):
    kind = s["kind"]
    if own:
        import log_linear_attention_fwd_gb300 as LL
        if kind == "glr_fwd":
            y = LL.loglinear_glr_fwd(s["x"], s["log_a"], h0=s["h0_"], cu_seqlens=s["cu"], scale=s["scale"], state=s["state"])
            return {"out": y, "state": s["state"]}
        if kind == "glr_bwd":
            dx, dla, dh0 = LL.loglinear_glr_bwd(s["x"], s["log_a"], s["out"], s["dout"], h0=s["h0_"], dstate=s["dstate"], cu_seqlens=s["cu"], scale=s["scale"])
            return {"dx": dx, "dlog_a": dla, "dh0": dh0}
        if kind == "glr_step":
            y = LL.loglinear_glr_step(s["state"], s["x"], s["log_a"], slots=s["slots"], scale=s["scale"])
            return {"out": y, "state": s["state"]}
        c = s["cache"]
        h = s.get("handle")
        if h is None:
            h = s["handle"] = LL.LogLinearCache(**c)
        if kind == "cache_step":
            LL.loglinear_cache_reserve(h, s["slots"], s["pos"])
            LL.loglinear_cache_step(h, s["slots"], s["pos"], s["q"], s["k"], s["v"], s["log_a"], s["lam"], out=s["out"])
            return {"out": s["out"], **c}
        if kind == "cache_load":
            a = s["a"]
            LL.loglinear_cache_load(h, a["slots"], s["T"], a["state"], a["k"], a["v"], a["log_a"])
            return dict(c)
        if kind == "cache_store":
            LL.loglinear_cache_store(h, s["slots"], s["pos"], s["dense"])
            return {"state": s["dense"]}
        if kind == "cache_fork":
            LL.loglinear_cache_fork(h, s["src"], s["dst"], s["pos"])
            return {k: c[k] for k in c if k != "pages"}
        live = []
        for one in (s["a"], s["b"]):
            LL.loglinear_cache_free(h, one["slots"])
            live.append(LL.loglinear_cache_compact(h))
            LL.loglinear_cache_load(h, one["slots"], s["T"], one["state"], one["k"], one["v"], one["log_a"])
        return {"live": live, **c}
    if kind == "glr_fwd":
        y, fin = _glr_fwd(s["x"].float(), s["log_a"].float(), s["h0_"], s["cu"], s["scale"])
        return {"out": y.to(s["x"].dtype), "state": fin}
    if kind == "glr_bwd":
        dx, dla, dh0 = _glr_bwd(s["x"].float(), s["log_a"].float(), s["out"].float(), s["dout"].float(), s["h0_"], s["dstate"], s["cu"], s["scale"])
        return {"dx": dx.to(s["dout"].dtype), "dlog_a": dla.to(s["log_a"].dtype), "dh0": dh0}
    if kind == "glr_step":
        la, at = s["log_a"].float(), s["slots"].long()
        h = torch.exp(la) * s["state"][at] + _scale(la, s["scale"])[0] * s["x"].float()
        s["state"][at] = h
        return {"out": h.to(s["x"].dtype), "state": s["state"]}
    c = s["cache"]
    if kind == "cache_step":
        _reserve(c, s["slots"], s["pos"])
        _step(c, s)
        return {"out": s["out"], **c}
    if kind == "cache_load":
        _load(c, s["a"], s["T"])
        return dict(c)
    if kind == "cache_store":
        _store(c, s["slots"].long(), s["pos"].long(), s["dense"])
        return {"state": s["dense"]}
    if kind == "cache_fork":
        _fork(c, s["src"].long(), s["dst"].long(), s["pos"].long())
        return {k: c[k] for k in c if k != "pages"}
    live = []
    for one in (s["a"], s["b"]):
        _release(c, one["slots"].long(), torch.zeros(len(one["slots"]), dtype=torch.int64, device="cuda"))
        live.append(_compact(c))
        _load(c, one, s["T"])
    return {"live": live, **c}


# ---------------------------------------------------------------------------- plain forms

def _scale(la, scale):
    """b(log a) and its derivative."""
    if scale == "none":
        return torch.ones_like(la), torch.zeros_like(la)
    if scale == "one_minus":
        return -torch.expm1(la), -torch.exp(la)
    b = torch.sqrt(-torch.expm1(2 * la))
    return b, torch.where(b > 0, -torch.exp(2 * la) / b, torch.zeros_like(b))


def _scan(a, u):
    """y_t = a_t y_{t-1} + u_t along dim 1, by doubling."""
    d, T = 1, a.shape[1]
    while d < T:
        u = torch.cat([u[:, :d], u[:, d:] + a[:, d:] * u[:, :-d]], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return u


def _bounds(cu, B, T):
    """For each position its sequence, whether it is the first and the last of it; for each
    sequence whether it is empty and its last position."""
    if cu is None:
        t = torch.arange(T, device="cuda").expand(B, T)
        seq = torch.arange(B, device="cuda")[:, None].expand(B, T)
        return seq, t == 0, t == T - 1, torch.zeros(B, dtype=torch.bool, device="cuda")
    cu = cu.long()
    t = torch.arange(T, device="cuda")
    seq = torch.searchsorted(cu, t, right=True) - 1
    return seq[None], (t == cu[seq])[None], (t == cu[seq + 1] - 1)[None], cu[1:] == cu[:-1]


def _glr_fwd(x, la, h0, cu, scale):
    B, T, D = x.shape
    seq, first, last, empty = _bounds(cu, B, T)
    a, u = torch.exp(la), _scale(la, scale)[0] * x
    if h0 is not None:
        u = u + first[..., None] * a * h0[seq]
    h = _scan(torch.where(first[..., None], torch.zeros_like(a), a), u)
    n = B if cu is None else cu.numel() - 1
    fin = torch.zeros(n, D, device="cuda") if h0 is None else h0.clone()
    fin[seq[last]] = h[last]
    return h, fin


def _glr_bwd(x, la, h, dout, h0, dstate, cu, scale):
    B, T, D = x.shape
    seq, first, last, empty = _bounds(cu, B, T)
    a = torch.exp(la)
    b, db = _scale(la, scale)
    u = dout if dstate is None else dout + last[..., None] * dstate[seq]
    c = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    c = torch.where(last[..., None], torch.zeros_like(c), c)
    g = _scan(c.flip(1), u.flip(1)).flip(1)
    before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    start = torch.zeros_like(h) if h0 is None else h0[seq]
    before = torch.where(first[..., None], start, before)
    dla = a * before * g + db * x * g
    dh0 = None
    if h0 is not None:
        dh0 = dstate.clone()
        dh0[seq[first]] = (a * g)[first]
    return b * g, dla, dh0


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


def _reserve(c, slots, pos):
    on = slots >= 0
    at, t = slots[on].long(), pos[on].long()
    j, end = t >> LOGW, t & (W - 1) == W - 1
    to = _ctz(j + 1)
    keep = j | torch.where(end, 1 << to, torch.zeros_like(to))
    _release(c, at, keep)
    m = torch.arange(c["page_table"].shape[1], device="cuda")
    _take(c, at, end[:, None] & (m == to[:, None]) & (c["page_table"][at] < 0))


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


def _window(c, at, H):
    k = c["win_k"][at].float().repeat_interleave(H // c["win_k"].shape[1], 1)
    return k, c["win_v"][at].float()


def _step(c, s):
    on = (s["slots"] >= 0).nonzero()[:, 0]
    at, t = s["slots"][on].long(), s["pos"][on].long()
    H, G = s["v"].shape[1], s["v"].shape[1] // s["k"].shape[1]
    M = s["M"]
    j, r = t >> LOGW, t & (W - 1)
    q, k = (s[x][on].float().repeat_interleave(G, 1) for x in ("q", "k"))
    v, lam = s["v"][on].float(), s["lam"][on]
    la = s["log_a"][on] if s["log_a"] is not None else torch.zeros(len(on), H, device="cuda")
    tok, page = _decays(c, at, t)
    tok, page = tok + la[..., None], page + la[:, None]
    wk, wv = _window(c, at, H)
    i = torch.arange(W, device="cuda")
    inside = (i < r[:, None])[:, None]
    lev = _bit_length(i ^ r[:, None])[:, None].expand(-1, H, -1)
    e = torch.where(inside, torch.exp(tok), torch.zeros_like(tok))
    p = torch.where(inside, lam.gather(2, lev) * e * (wk * q[:, :, None]).sum(-1), torch.zeros_like(tok))
    o = torch.where(inside[..., None], p[..., None] * wv, torch.zeros_like(wv)).sum(2)
    o = o + (lam[..., 0] * (q * k).sum(-1))[..., None] * v
    m = torch.arange(M, device="cuda")
    live = ((j[:, None] >> m) & 1 == 1)[..., None]
    ep = torch.where(live, torch.exp(page), torch.zeros_like(page))
    held = c["pages"][c["page_table"][at].clamp(min=0).long()]      # [n, M, H, dk, dv]
    w = ep * lam[..., LOGW + 1:LOGW + 1 + M].transpose(1, 2)
    o = o + (w[..., None] * torch.matmul(q[:, None, :, None], held)[..., 0, :]).sum(1)
    s["out"][on] = o.to(s["out"].dtype)
    f = (r == W - 1).nonzero()[:, 0]                                # blocks that end here
    to = _ctz(j[f] + 1)
    low = (m < to[:, None])[..., None] * ep[f]
    new = (low[..., None, None] * held[f]).sum(1)
    new = new + torch.matmul((e[f][..., None] * wk[f])[:, :, :W - 1].transpose(2, 3), wv[f][:, :, :W - 1])
    new = new + k[f][..., None] * v[f][:, :, None]
    c["pages"][c["page_table"][at[f], to].long()] = new
    c["win_k"][at, :, r], c["win_v"][at, :, r] = s["k"][on], s["v"][on]
    c["win_log_a"][at, :, r] = la
    after = (j[f] + 1)[:, None] >> m & 1 == 1
    log = torch.where((m == to[:, None])[..., None], torch.zeros_like(page[f]), page[f])
    old = c["page_log"][at[f], (j[f] + 1) & 1]
    c["page_log"][at[f], (j[f] + 1) & 1] = torch.where(after[..., None], log, old)
    c["page_from"][at[f], (j[f] + 1) & 1] = 0


def _load(c, one, T):
    at = one["slots"].long()
    n, M = len(at), c["page_table"].shape[1]
    _release(c, at, torch.zeros_like(at))
    j, r = T >> LOGW, T & (W - 1)
    bits = [i for i in range(M) if j >> i & 1]
    _take(c, at, torch.tensor([i in bits for i in range(M)], device="cuda").expand(n, M))
    st = one["state"]
    for i in bits:
        level = st[:, :, LOGW + 1 + i]
        if r == 0 and i == bits[0]:  # the block ended with the prompt: its levels become one page
            level = st[:, :, :LOGW + 1 + i].sum(2)
        c["pages"][c["page_table"][at, i].long()] = level
        c["page_log"][at, j & 1, i] = 0.0
    c["page_from"][at, j & 1] = r
    if r:
        c["win_k"][at, :, :r] = one["k"][:, -r:].transpose(1, 2)
        c["win_v"][at, :, :r] = one["v"][:, -r:].transpose(1, 2)
        c["win_log_a"][at, :, :r] = one["log_a"][:, -r:].transpose(1, 2)


def _store(c, at, n, dense):
    """Dense states after n positions.  Where a block has just ended, the levels that the next
    step merges come as their sum, in the highest of them."""
    H, L, M = dense.shape[1], dense.shape[2], c["page_table"].shape[1]
    dense.zero_()
    j, r = n >> LOGW, n & (W - 1)
    tok, page = _decays(c, at, n)
    i = torch.arange(W, device="cuda")
    lev = _bit_length(i ^ (r - 1).clamp(min=0)[:, None])
    e = torch.where((i < r[:, None])[:, None], torch.exp(tok), torch.zeros_like(tok))
    wk, wv = _window(c, at, H)
    wv = torch.where((i < r[:, None])[:, None, :, None], wv, torch.zeros_like(wv))
    one = (lev[:, None] == torch.arange(LOGW + 1, device="cuda")[:, None]).float()   # [n, 7, W]
    k2 = one[:, None, :, :, None] * (e[..., None] * wk)[:, :, None]                   # [n, H, 7, W, dk]
    dense[:, :, :LOGW + 1] = torch.matmul(k2.transpose(3, 4), wv[:, :, None])
    m = torch.arange(M, device="cuda")
    live = ((j[:, None] >> m) & 1 == 1)[..., None]
    ep = torch.where(live, torch.exp(page), torch.zeros_like(page))
    held = ep[..., None, None] * c["pages"][c["page_table"][at].clamp(min=0).long()]
    sums = torch.where((r == 0)[:, None] & (m == _ctz(j)[:, None]), LOGW + m, LOGW + 1 + m)   # level of each page
    row, col = live[..., 0].nonzero(as_tuple=True)
    dense[row, :, sums[row, col]] = held[row, col]


def _fork(c, src, dst, pos):
    _release(c, dst, torch.zeros_like(dst))
    j, r = pos >> LOGW, pos & (W - 1)
    live = (j[:, None] >> torch.arange(c["page_table"].shape[1], device="cuda")) & 1 == 1
    row = torch.where(live, c["page_table"][src], torch.full_like(c["page_table"][src], NEG))
    c["page_table"][dst] = row
    c["refcount"].index_add_(0, row[live].long(), torch.ones(int(live.sum()), dtype=torch.int32, device="cuda"))
    inside = torch.arange(W, device="cuda") < r[:, None]
    for name, mask in (("win_k", inside[:, None, :, None]), ("win_v", inside[:, None, :, None]), ("win_log_a", inside[:, None])):
        c[name][dst] = torch.where(mask, c[name][src], c[name][dst])
    c["page_log"][dst, j & 1] = torch.where(live[..., None], c["page_log"][src, j & 1], c["page_log"][dst, j & 1])
    c["page_from"][dst, j & 1] = c["page_from"][src, j & 1]


def _compact(c):
    used = c["refcount"] > 0
    live = int(used.sum())
    high, low = used[live:].nonzero()[:, 0] + live, (~used[:live]).nonzero()[:, 0]
    c["pages"][low] = c["pages"][high]
    to = torch.arange(used.numel(), device="cuda")
    to[high] = low
    t = c["page_table"]
    t.copy_(torch.where(t >= 0, to[t.clamp(min=0).long()].to(torch.int32), t))
    c["refcount"][low] = c["refcount"][high]
    c["refcount"][high] = 0
    return torch.full((1,), live, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------- what a pass needs

def work(c):
    size = {"f32": 4, "bf16": 2}
    kind, e = c["kind"], {"f32": 4, "bf16": 2}[c["dtype"]]
    if kind.startswith("glr"):
        g, D = size[c["gate"]], c["D"]
        if kind == "glr_step":
            return {"bytes": c["B"] * D * (2 * e + g + 8), "flops": 8 * c["B"] * D}
        n, rows = c["N"] or c["B"], c["B"] * c["T"] * D
        if kind == "glr_fwd":
            return {"bytes": rows * (2 * e + g) + n * D * (8 if c["h0"] else 4), "flops": 8 * rows}
        per = 3 * e + 2 * g + (e if c["scale"] != "none" else 0)
        return {"bytes": rows * per + (12 * n * D if c["h0"] else 0), "flops": 16 * rows}
    H, Hqk, dk, dv = c["H"], c["Hqk"], c["dk"], c["dv"]
    page, token = 4 * H * dk * dv, e * (Hqk * dk + H * dv) + 4 * H
    if kind == "cache_step":
        b = f = 0
        for p in _positions(c, c["B"])[:c["B"] - c["pad"]]:
            j, r = p >> LOGW, p & (W - 1)
            b += page * (bin(j).count("1") + (r == W - 1)) + token * (r + 2) + e * (Hqk * dk + H * dv) + 4 * H * (r.bit_length() + 1)
            f += 2 * H * dk * dv * (bin(j).count("1") + (W if r == W - 1 else 0)) + 2 * H * r * (dk + dv)
        return {"bytes": b, "flops": f}
    if kind in ("cache_load", "cache_churn"):
        j, r = c["T"] >> LOGW, c["T"] & (W - 1)
        p = bin(j).count("1")
        more = (LOGW + (j & -j).bit_length() - 1) if r == 0 and j else 0
        one = c["n"] * (page * (2 * p + more) + 2 * token * r)
        return {"bytes": one if kind == "cache_load" else 2 * one + 4 * c["n"] * page * p, "flops": c["n"] * page // 4 * more}
    pos = _positions(c, c["n"])
    if kind == "cache_store":
        L = LOGW + 1 + _levels(c["hi"])
        return {"bytes": sum(page * (bin(p >> LOGW).count("1") + L) + token * (p & (W - 1)) for p in pos), "flops": sum(2 * H * dk * dv * (p & (W - 1)) for p in pos)}
    return {"bytes": c["copies"] * sum(2 * token * (p & (W - 1)) + 8 * H * bin(p >> LOGW).count("1") for p in pos) + 64, "flops": 0}


# ---------------------------------------------------------------------------- 64 bits

def exact(c, seed):
    """run()'s values in 64 bits: the recurrence token by token; the cache operators sequence by sequence."""
    s = prepare(c, seed)
    kind = c["kind"]
    if kind in ("glr_fwd", "glr_bwd"):
        return _exact_glr(c, s)
    if kind == "glr_step":
        la, at = s["log_a"].double(), s["slots"].long()
        b = {"none": torch.ones_like(la), "one_minus": 1 - la.exp(), "sqrt": (1 - (2 * la).exp()).clamp(min=0).sqrt()}[c["scale"]]
        st = s["state"].double()
        st[at] = la.exp() * st[at] + b * s["x"].double()
        return {"out": st[at], "state": st}
    if kind == "cache_step":
        return _exact_step(c, s)
    if kind == "cache_store":
        return {"state": _exact_store(c, s)}
    return None  # copies and sums of a few fp32 values, at places that the tables give


def _exact_glr(c, s):
    B, T, D = s["x"].shape
    la, x = s["log_a"].double(), s["x"].double()
    a = la.exp()
    b = {"none": torch.ones_like(la), "one_minus": 1 - a, "sqrt": (1 - a * a).clamp(min=0).sqrt()}[c["scale"]]
    cu = _cuts(c) if c["N"] else None
    spans = [(0, cu[i], cu[i + 1], i) for i in range(c["N"])] if cu else [(0, 0, T, slice(0, B))]
    rows = slice(0, B)
    n = c["N"] or B
    zero = torch.zeros(n, D, dtype=torch.float64, device="cuda")
    h0 = zero if s["h0_"] is None else s["h0_"].double()
    if c["kind"] == "glr_fwd":
        out, fin = torch.zeros(B, T, D, dtype=torch.float64, device="cuda"), h0.clone()
        bx = b * x
        for _, lo, hi, i in spans:
            h = h0[i]
            for t in range(lo, hi):
                h = torch.addcmul(bx[rows, t], a[rows, t], h)
                out[rows, t] = h
            if hi > lo:
                fin[i] = h if not isinstance(i, int) else h[0]
        return {"out": out, "state": fin}
    h, dout = s["out"].double(), s["dout"].double()
    g = torch.zeros_like(dout)
    before = torch.zeros_like(dout)
    dh0 = zero.clone() if s["dstate"] is None else s["dstate"].double()
    for _, lo, hi, i in spans:
        if hi == lo:
            continue
        before[rows, lo + 1:hi] = h[rows, lo:hi - 1]
        before[rows, lo] = h0[i]
        carry = dh0[i]
        for t in range(hi - 1, lo - 1, -1):
            carry = dout[rows, t] + carry
            g[rows, t] = carry
            carry = a[rows, t] * carry
        dh0[i] = carry if not isinstance(i, int) else carry[0]
    db = {"none": torch.zeros_like(la), "one_minus": -a, "sqrt": torch.where(b > 0, -a * a / b, torch.zeros_like(b))}[c["scale"]]
    return {"dx": b * g, "dlog_a": a * before * g + db * x * g, "dh0": dh0 if s["h0_"] is not None else None}


def _exact_step(c, s):
    cache = s["cache"]
    _reserve(cache, s["slots"], s["pos"])  # whole numbers; no values come of it
    out = s["out"].double()
    new = {k: cache[k].double() for k in ("pages", "win_k", "win_v", "win_log_a", "page_log")}
    pages = cache["pages"].double()
    H, G = c["H"], c["H"] // c["Hqk"]
    for row, (slot, t) in enumerate(zip(s["slots"].tolist(), s["pos"].tolist())):
        if slot < 0:
            continue
        q, k = (s[x][row].double().repeat_interleave(G, 0) for x in ("q", "k"))
        v, lam = s["v"][row].double(), s["lam"][row].double()
        la = s["log_a"][row].double() if s["log_a"] is not None else torch.zeros(H, dtype=torch.float64, device="cuda")
        j, r = t // W, t % W
        las = torch.cat([cache["win_log_a"][slot, :, :r].double(), la[:, None]], 1)     # [H, r + 1]
        ks = torch.cat([cache["win_k"][slot, :, :r].double().repeat_interleave(G, 0), k[:, None]], 1)
        vs = torch.cat([cache["win_v"][slot, :, :r].double(), v[:, None]], 1)
        dec = torch.stack([las[:, i + 1:].sum(1) for i in range(r + 1)], 1).exp()
        lv = torch.tensor([(i ^ r).bit_length() for i in range(r + 1)], device="cuda")
        o = (((ks * q[:, None]).sum(-1) * dec * lam[:, lv])[..., None] * vs).sum(1)
        fold = torch.zeros(H, c["dk"], c["dv"], dtype=torch.float64, device="cuda")
        to = ((j + 1) & -(j + 1)).bit_length() - 1
        since = las[:, int(cache["page_from"][slot, j & 1]):].sum(1)
        for i in range(s["M"]):
            if j >> i & 1:
                log = cache["page_log"][slot, j & 1, i].double() + since
                P = log.exp()[:, None, None] * pages[int(cache["page_table"][slot, i])]
                o = o + lam[:, LOGW + 1 + i, None] * torch.einsum("hd,hde->he", q, P)
                if i < to:
                    fold = fold + P
                elif r == W - 1:
                    new["page_log"][slot, (j + 1) & 1, i] = log
        out[row] = o
        if r == W - 1:
            new["pages"][int(cache["page_table"][slot, to])] = fold + torch.einsum("hsd,hse->hde", dec[..., None] * ks, vs)
            new["page_log"][slot, (j + 1) & 1, to] = 0
        new["win_k"][slot, :, r], new["win_v"][slot, :, r], new["win_log_a"][slot, :, r] = s["k"][row].double(), v, la
    return {"out": out, **{k: new.get(k) for k in cache}}


def _exact_store(c, s):
    cache, G = s["cache"], c["H"] // c["Hqk"]
    dense = torch.zeros(s["dense"].shape, dtype=torch.float64, device="cuda")
    for row, (slot, n) in enumerate(zip(s["slots"].tolist(), s["pos"].tolist())):
        j, r = n // W, n % W
        la = cache["win_log_a"][slot, :, :r].double()
        for i in range(r):
            k = cache["win_k"][slot, :, i].double().repeat_interleave(G, 0) * la[:, i + 1:].sum(1).exp()[:, None]
            dense[row, :, (i ^ (r - 1)).bit_length()] += k[..., None] * cache["win_v"][slot, :, i].double()[:, None]
        since = la[:, int(cache["page_from"][slot, j & 1]):].sum(1)
        for i in range(s["M"]):
            if j >> i & 1:
                level = LOGW + i if r == 0 and j & ((1 << i) - 1) == 0 else LOGW + 1 + i
                log = cache["page_log"][slot, j & 1, i].double() + since
                dense[row, :, level] = log.exp()[:, None, None] * cache["pages"][int(cache["page_table"][slot, i])].double()
    return dense
