"""The gated linear recurrence on the GPU against its fp64 oracle.

fp32 results: a gate is off by at most 2^-22 relative, a token's weight after k steps by k
times that, independently per step; with 1 - a >= 0.01 (k up to about 100) that is about
sqrt(100) * 2^-22 = 2.4e-6 of the state, and 1e-5 (TOL_F32) bounds it.  bf16 results add half a
step of the type, 2^-8 of each value.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
from tests.helpers import TOL_F32, rel_l2, to64

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def LL():
    import log_linear_attention_fwd_gb300 as m
    return m


def make(B, T, D, dtype="f32", gate="f32", seed=0, lo=-1.5, hi=-0.01):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, T, D, generator=g).to(DT[dtype])
    la = (lo + (hi - lo) * torch.rand(B, T, D, generator=g)).to(DT[gate])
    return x, la


def dev(*ts):
    return [None if t is None else t.cuda() for t in ts]


def check(got, want, what=""):
    """fp32: rel-L2; bf16: every value within half a step plus the fp32 error."""
    if got.numel() == 0:
        return
    if got.dtype == torch.float32:
        assert rel_l2(got, want) <= TOL_F32, (what, rel_l2(got, want))
    else:
        rms = float(np.sqrt(np.mean(np.square(want))))
        off = np.abs(to64(got) - want) - (2.0 ** -8 * np.abs(want) + TOL_F32 * rms)
        assert off.max() <= 0, (what, off.max())


def fwd_bwd(LL, x, la, scale, h0=None, cu=None, dout=None, ds=None, out_dtype=None):
    """Forward and backward on the GPU against the oracle."""
    B, T, D = la.shape
    n = B if cu is None else len(cu) - 1
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32).cuda()
    xd, ld, hd, dd, sd = dev(x, la, h0, dout, ds)
    state = torch.full((n, D), float("nan")).cuda()
    out = LL.loglinear_glr_fwd(xd, ld, h0=hd, cu_seqlens=c, scale=scale, state=state,
                               out_dtype=out_dtype)
    want, last = oracle.glr_forward(x, la, scale, h0=h0, cu=cu)
    on = ~np.isnan(want)
    check(out.cpu()[torch.from_numpy(on)], want[on], "out")
    check(state.cpu(), last, "state")
    grads = LL.loglinear_glr_bwd(xd, ld, out, dd.to(out.dtype), h0=hd, cu_seqlens=c, scale=scale, dstate=sd)
    wants = oracle.glr_backward(x, la, out, dd.to(out.dtype), scale, h0=h0, dstate=ds, cu=cu)
    for name, g, w in zip(("dx", "dlog_a", "dh0"), grads, wants):
        if g is None:
            continue
        on = ~np.isnan(w)
        check(g.cpu()[torch.from_numpy(on)], w[on], name)
    torch.cuda.synchronize()
    return out, state, grads


@pytest.mark.parametrize("scale", ["none", "one_minus", "sqrt"])
@pytest.mark.parametrize("dtype,gate", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("B,T,D", [(1, 1, 1), (2, 63, 2), (1, 64, 64), (3, 65, 66), (1, 127, 31),
                                   (2, 130, 130), (1, 1100, 40), (1, 2049, 8)])
def test_sizes(LL, B, T, D, dtype, gate, scale):
    x, la = make(B, T, D, dtype, gate, seed=T)
    g = torch.Generator().manual_seed(5)
    fwd_bwd(LL, x, la, scale, dout=torch.randn(B, T, D, generator=g))
    h0, ds = torch.randn(B, D, generator=g), torch.randn(B, D, generator=g)
    fwd_bwd(LL, x, la, scale, h0=h0, dout=torch.randn(B, T, D, generator=g), ds=ds)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_out_dtypes(LL, dtype, out_dtype):
    x, la = make(2, 300, 72, dtype, "f32", seed=3)
    dout = torch.randn(2, 300, 72, generator=torch.Generator().manual_seed(4))
    out, _, (dx, dla, _) = fwd_bwd(LL, x, la, "sqrt", dout=dout, out_dtype=out_dtype)
    assert out.dtype == dx.dtype == out_dtype and dla.dtype == torch.float32


@pytest.mark.parametrize("cu", [[0, 300], [0, 0, 1, 2, 2, 2, 130, 131, 300], [0, 64, 128, 128, 200],
                                [0, 0, 0], [0, 299, 299, 299]])
@pytest.mark.parametrize("dtype,D", [("f32", 66), ("bf16", 24), ("f32", 5)])
@pytest.mark.parametrize("scale", ["none", "sqrt"])
def test_packed(LL, cu, dtype, D, scale):
    T, n = 300, len(cu) - 1
    x, la = make(1, T, D, dtype, "f32", seed=n)
    g = torch.Generator().manual_seed(6)
    h0, ds = torch.randn(n, D, generator=g), torch.randn(n, D, generator=g)
    dout = torch.randn(1, T, D, generator=g)
    fwd_bwd(LL, x, la, scale, h0=h0, cu=cu, dout=dout, ds=ds)
    fwd_bwd(LL, x, la, scale, cu=cu, dout=dout)


def test_many_short_sequences(LL):
    """Several sequences inside one warp's tokens, and more sequences than warps."""
    lens = [1, 2, 3, 0, 0, 5, 1, 1, 1, 0, 7, 2] * 40
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    x, la = make(1, cu[-1], 10, seed=9)
    g = torch.Generator().manual_seed(6)
    n = len(lens)
    fwd_bwd(LL, x, la, "one_minus", h0=torch.randn(n, 10, generator=g), cu=cu,
            dout=torch.randn(1, cu[-1], 10, generator=g), ds=torch.randn(n, 10, generator=g))


def test_rows_behind_the_last_sequence_stay(LL):
    T, D, cu = 200, 12, torch.tensor([0, 30, 77], dtype=torch.int32).cuda()
    x, la = make(1, T, D)
    x[:, 77:] = float("nan")
    la[:, 77:] = float("nan")
    out = torch.full((1, T, D), 7.0).cuda()
    LL.loglinear_glr_fwd(x.cuda(), la.cuda(), cu_seqlens=cu, out=out)
    assert torch.all(out[:, 77:] == 7) and torch.isfinite(out).all()
    want, _ = oracle.glr_forward(x[:, :77], la[:, :77], cu=[0, 30, 77])
    check(out[:, :77].cpu(), want)


def test_nothing_passes_between_sequences(LL):
    """Infinities and NaN of one sequence stay there, forward and backward."""
    T, D, cu = 400, 6, [0, 100, 210, 400]
    x, la = make(1, T, D, seed=2)
    x[0, 150], x[0, 151] = float("inf"), float("nan")
    g = torch.Generator().manual_seed(1)
    dout = torch.randn(1, T, D, generator=g)
    dout[0, 160], dout[0, 161] = float("inf"), float("nan")
    c = torch.tensor(cu, dtype=torch.int32).cuda()
    out = LL.loglinear_glr_fwd(x.cuda(), la.cuda(), cu_seqlens=c, scale="sqrt")
    dx, dla, _ = LL.loglinear_glr_bwd(x.cuda(), la.cuda(), out, dout.cuda(), cu_seqlens=c, scale="sqrt")
    assert torch.isnan(out[0, 151:210]).all() and not torch.isfinite(dx[0, 100:162]).any()
    for lo, hi in ((0, 100), (210, 400)):
        want, _ = oracle.glr_forward(x[:, lo:hi], la[:, lo:hi], "sqrt")
        check(out[:, lo:hi].cpu(), want)
        w = oracle.glr_backward(x[:, lo:hi], la[:, lo:hi], out[:, lo:hi], dout[:, lo:hi], "sqrt")
        check(dx[:, lo:hi].cpu(), w[0])
        check(dla[:, lo:hi].cpu(), w[1])


@pytest.mark.parametrize("scale", ["none", "one_minus", "sqrt"])
def test_extreme_gates(LL, scale):
    """log a of 0 (a = 1), tiny, -inf and the type's lowest value."""
    B, T, D = 1, 200, 16
    x, la = make(B, T, D, seed=8)
    la[0, 10:20], la[0, 40], la[0, 90:95] = 0.0, -float("inf"), torch.finfo(torch.float32).min
    la[0, 120:125], la[0, 140:150] = -1e-7, -60.0
    la[0, 160:170] = torch.linspace(-0.6, -0.4, 10)[:, None]
    g = torch.Generator().manual_seed(1)
    # near a = 1 the derivative of the square root is about -1 / b; the oracle has it too
    fwd_bwd(LL, x, la, scale, dout=torch.randn(B, T, D, generator=g), h0=torch.randn(B, D, generator=g))


def test_gate_accuracy_near_one(LL):
    """b keeps its relative accuracy where a rounds to 1: |log a| down to 2^-30."""
    la = -torch.exp2(-torch.arange(1, 31, dtype=torch.float64)).float().reshape(1, 30, 1)
    x = torch.ones(1, 30, 1)
    for scale in ("one_minus", "sqrt"):
        cu = torch.arange(31, dtype=torch.int32).cuda()   # one token per sequence: h = b
        got = LL.loglinear_glr_fwd(x.cuda(), la.cuda(), cu_seqlens=cu, scale=scale).cpu()
        want, _ = oracle.glr_scale(la, scale)
        assert np.max(np.abs(to64(got) / want - 1)) <= 2.0 ** -21  # sqrt and exp: 2^-22 each


def test_long_sums_are_exact(LL):
    """a = 1, small integers: any order of fp32 sums is exact, across all tiles and CTAs."""
    for T, D in ((20000, 3), (5000, 130)):
        g = torch.Generator().manual_seed(T)
        x = torch.randint(-2, 3, (1, T, D), generator=g).float()
        la = torch.zeros(1, T, D)
        out = LL.loglinear_glr_fwd(x.cuda(), la.cuda())
        assert torch.equal(out.cpu(), x.cumsum(1))
        dx, _, _ = LL.loglinear_glr_bwd(None, la.cuda(), out, x.cuda())
        assert torch.equal(dx.cpu(), x.flip(1).cumsum(1).flip(1))


def test_clusters_of_odd_sizes_are_exact(LL):
    """As above, where a channel block's CTAs are not a power of two, and packed."""
    for T, D in ((1300, 40), (2500, 514), (9001, 1000)):
        g = torch.Generator().manual_seed(T)
        x = torch.randint(-2, 3, (1, T, D), generator=g).float()
        la = torch.zeros(1, T, D)
        h0 = torch.randint(-9, 10, (3, D), generator=g).float()
        cu = [0, T // 3, T // 2 + 1, T]
        c = torch.tensor(cu, dtype=torch.int32).cuda()
        state = torch.empty(3, D).cuda()
        out = LL.loglinear_glr_fwd(x.cuda(), la.cuda(), h0=h0.cuda(), cu_seqlens=c, state=state)
        dx, _, dh0 = LL.loglinear_glr_bwd(None, la.cuda(), out, x.cuda(), h0=h0.cuda(), cu_seqlens=c,
                                          dstate=h0.cuda())
        for n, (lo, hi) in enumerate(zip(cu, cu[1:])):
            want = x[0, lo:hi].cumsum(0) + h0[n]
            assert torch.equal(out[0, lo:hi].cpu(), want) and torch.equal(state[n].cpu(), want[-1])
            back = x[0, lo:hi].flip(0).cumsum(0).flip(0) + h0[n]
            assert torch.equal(dx[0, lo:hi].cpu(), back) and torch.equal(dh0[n].cpu(), back[0])


@pytest.mark.parametrize("n", [15, 16, 255, 256, 257])
def test_numbers_of_sequences(LL, n):
    """Around the counts at which the bounds are read from another place."""
    g = torch.Generator().manual_seed(n)
    lens = torch.randint(0, 6, (n,), generator=g)
    cu = np.concatenate([[0], np.cumsum(lens.numpy())]).tolist()
    T, D = cu[-1] + 3, 12
    x, la = make(1, T, D, seed=n)
    fwd_bwd(LL, x, la, "sqrt", h0=torch.randn(n, D, generator=g), cu=cu,
            dout=torch.randn(1, T, D, generator=g), ds=torch.randn(n, D, generator=g))


def test_first_call_inside_a_capture(LL):
    """What a call asks of the runtime the first time is allowed while a stream is captured."""
    code = """
import torch, log_linear_attention_fwd_gb300 as LL
x, la = torch.randn(1, 3000, 70).cuda(), -torch.rand(1, 3000, 70).cuda()
cu, out = torch.tensor([0, 5, 1000, 3000], dtype=torch.int32).cuda(), torch.empty_like(x)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    LL.loglinear_glr_fwd(x, la, out=out, scale="sqrt", cu_seqlens=cu)
    grads = LL.loglinear_glr_bwd(x, la, out, x, scale="sqrt", cu_seqlens=cu)
g.replay()
o = LL.loglinear_glr_fwd(x, la, scale="sqrt", cu_seqlens=cu)
want = LL.loglinear_glr_bwd(x, la, o, x, scale="sqrt", cu_seqlens=cu)
assert torch.equal(o, out) and all(torch.equal(a, b) for a, b in zip(grads[:2], want[:2]))
assert LL.device_error() == 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]


def test_results_do_not_depend_on_timing(LL):
    x, la = make(2, 6000, 192, "bf16", "f32", seed=4)
    dout = torch.randn(2, 6000, 192, generator=torch.Generator().manual_seed(4)).bfloat16()
    xd, ld, dd = dev(x, la, dout)
    one = LL.loglinear_glr_fwd(xd, ld, scale="sqrt")
    g1 = LL.loglinear_glr_bwd(xd, ld, one, dd, scale="sqrt")
    for _ in range(5):
        two = LL.loglinear_glr_fwd(xd, ld, scale="sqrt")
        g2 = LL.loglinear_glr_bwd(xd, ld, two, dd, scale="sqrt")
        assert torch.equal(one, two) and all(torch.equal(a, b) for a, b in zip(g1[:2], g2[:2]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 37])
def test_strided_and_unaligned(LL, dtype, D):
    """Slices of a fused projection, a batch broadcast, and pointers off by one element."""
    B, T = 2, 150
    fused = torch.randn(B, T, 2 * D + 1, generator=torch.Generator().manual_seed(1)).to(DT[dtype])
    fused[..., D + 1:] = -0.05 - torch.rand(B, T, D).to(DT[dtype])
    f = fused.cuda()
    x, la = f[..., 1:D + 1], f[..., D + 1:]
    want, _ = oracle.glr_forward(x, la, "sqrt")
    out = LL.loglinear_glr_fwd(x, la, scale="sqrt")
    check(out.cpu(), want)
    dout = torch.randn(B, T, D, generator=torch.Generator().manual_seed(2)).to(DT[dtype])
    got = LL.loglinear_glr_bwd(x, la, out, dout.cuda(), scale="sqrt")
    for g, w in zip(got, oracle.glr_backward(x, la, out, dout, "sqrt")):
        if g is not None:
            check(g.cpu(), w)
    one = la[:1].expand(B, T, D)   # batch stride 0
    want, _ = oracle.glr_forward(x, one, "none")
    check(LL.loglinear_glr_fwd(x, one, scale="none").cpu(), want)
    buf = torch.empty(B * T * D + 1, dtype=DT[dtype]).cuda()
    o = buf[1:].view(B, T, D)
    LL.loglinear_glr_fwd(x, la, scale="sqrt", out=o)
    assert torch.equal(o, out)


def test_empty_calls(LL):
    h0 = torch.randn(2, 5).cuda()
    state = torch.zeros(2, 5).cuda()
    e = torch.empty(2, 0, 5).cuda()
    LL.loglinear_glr_fwd(e, e, h0=h0, state=state)
    assert torch.equal(state, h0)
    dx, dla, dh0 = LL.loglinear_glr_bwd(e, e, e, e, h0=h0, dstate=state)
    assert dx.shape == (2, 0, 5) and torch.equal(dh0, state)
    assert LL.loglinear_glr_fwd(torch.empty(0, 4, 5).cuda(), torch.empty(0, 4, 5).cuda()).numel() == 0
    cu = torch.zeros(1, dtype=torch.int32).cuda()       # no sequences
    out = torch.full((1, 4, 5), 3.0).cuda()
    LL.loglinear_glr_fwd(torch.zeros(1, 4, 5).cuda(), torch.zeros(1, 4, 5).cuda(), cu_seqlens=cu, out=out)
    assert torch.all(out == 3)


def test_malformed_bounds_stay_inside(LL):
    """Bounds out of order or past T: wrong sequences, but finite work and no access outside."""
    x, la = make(1, 100, 8)
    pad = torch.full((300, 8), 9.0).cuda()
    out = pad[100:200].view(1, 100, 8)
    for bounds in ([0, 50, 20, 500], [-7, 30, 90], [200, 300], [90, 10, 0]):
        cu = torch.tensor(bounds, dtype=torch.int32).cuda()
        n = len(bounds) - 1
        state = torch.full((n + 2, 8), 9.0).cuda()
        LL.loglinear_glr_fwd(x.cuda(), la.cuda(), cu_seqlens=cu, out=out, state=state[1:n + 1])
        torch.cuda.synchronize()
        assert torch.all(pad[:100] == 9) and torch.all(pad[200:] == 9)
        assert torch.all(state[0] == 9) and torch.all(state[-1] == 9)


@pytest.mark.parametrize("D", [1, 2, 37, 64, 700])
@pytest.mark.parametrize("dtype,gate", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
def test_step_continues_the_forward(LL, D, dtype, gate):
    B, T = 3, 9
    x, la = make(B, T, D, dtype, gate, seed=D)
    want, last = oracle.glr_forward(x, la, "sqrt")
    xd, ld = dev(x, la)
    pool = torch.full((8, D), 5.0).cuda()
    slots = torch.tensor([6, 1, 3], dtype=torch.int32).cuda()
    state = torch.empty(B, D).cuda()
    LL.loglinear_glr_fwd(xd[:, :4].contiguous(), ld[:, :4].contiguous(), scale="sqrt", state=state)
    pool[slots.long()] = state
    for t in range(4, T):
        y = LL.loglinear_glr_step(pool, xd[:, t].contiguous(), ld[:, t].contiguous(), slots=slots, scale="sqrt")
        check(y.cpu(), want[:, t])
        LL.loglinear_glr_step(state, xd[:, t].contiguous(), ld[:, t].contiguous(), scale="sqrt")
    check(pool[slots.long()].cpu(), last)
    assert torch.equal(state, pool[slots.long()])
    assert torch.all(pool[[0, 2, 4, 5, 7]] == 5)
    assert LL.device_error() == 0


def test_step_bad_slots(LL):
    D = 40
    x, la = make(1, 6, D)
    pool = torch.arange(4.0)[:, None].expand(4, D).contiguous().cuda()
    keep = pool.clone()
    slots = torch.tensor([2, -1, 2, 4, -5, 0], dtype=torch.int32).cuda()
    out = torch.full((6, D), 9.0).cuda()
    LL.loglinear_glr_step(pool, x[0].cuda(), la[0].cuda(), slots=slots, out=out)
    assert LL.device_error() == 1 << 4 and LL.device_error() == 0
    assert torch.all(out[[1, 2, 3, 4]] == 9) and torch.equal(pool[[1, 3]], keep[[1, 3]])
    for row, slot in ((0, 2), (5, 0)):
        want = np.exp(to64(la[0, row])) * to64(keep[slot]) + to64(x[0, row])
        check(pool[slot].cpu(), want)
        assert torch.equal(pool[slot], out[row])
    # padding alone is no error
    LL.loglinear_glr_step(pool, x[0, :2].cuda(), la[0, :2].cuda(), slots=slots[:2].contiguous() * 0 - 1)
    assert LL.device_error() == 0


@pytest.mark.parametrize("T", [1, 700, 9000])
def test_states_in_place(LL, T):
    """The last states may go where the first ones are, and likewise their gradients."""
    x, la = dev(*make(2, T, 70, seed=T))
    h0 = torch.randn(2, 70, generator=torch.Generator().manual_seed(1)).cuda()
    state, both = torch.empty_like(h0), h0.clone()
    a = LL.loglinear_glr_fwd(x, la, h0=h0, state=state, scale="sqrt")
    b = LL.loglinear_glr_fwd(x, la, h0=both, state=both, scale="sqrt")
    assert torch.equal(a, b) and torch.equal(state, both)


def test_side_stream_and_graph(LL):
    x, la = dev(*make(2, 700, 96, "bf16", "f32", seed=12))
    want = LL.loglinear_glr_fwd(x, la, scale="sqrt")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = LL.loglinear_glr_fwd(x, la, scale="sqrt", stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out, state = torch.empty_like(want), torch.zeros(2, 96).cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        LL.loglinear_glr_fwd(x, la, scale="sqrt", out=out, state=state)
        dx, dla, _ = LL.loglinear_glr_bwd(x, la, out, x, scale="sqrt")
    x.copy_(x.flip(1))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, LL.loglinear_glr_fwd(x, la, scale="sqrt"))
    assert torch.equal(dx, LL.loglinear_glr_bwd(x, la, out, x, scale="sqrt")[0])


def test_headline_size(LL):
    """B1 T16384 D2048 bf16 on sampled channels (each channel is a problem of its own)."""
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(1, 16384, 2048, generator=g, device="cuda").bfloat16()
    la = -0.02 - torch.rand(1, 16384, 2048, generator=g, device="cuda")
    out = LL.loglinear_glr_fwd(x, la, scale="sqrt")
    dout = torch.randn(1, 16384, 2048, generator=g, device="cuda").bfloat16()
    dx, dla, _ = LL.loglinear_glr_bwd(x, la, out, dout, scale="sqrt")
    at = torch.tensor([0, 1, 63, 64, 777, 2047]).cuda()
    cut = lambda t: t[..., at].contiguous()  # noqa: E731
    want, _ = oracle.glr_forward(cut(x), cut(la), "sqrt")
    check(cut(out).cpu(), want)
    w = oracle.glr_backward(cut(x), cut(la), cut(out), cut(dout), "sqrt")
    check(cut(dx).cpu(), w[0])
    check(cut(dla).cpu(), w[1])


@pytest.mark.parametrize("la0", [-1.5, -60.0])
@pytest.mark.parametrize("T,D,packed", [(70, 3, False), (3000, 40, False), (700, 6, True)])
def test_infinite_states_stay_infinite(LL, la0, T, D, packed):
    """An infinity times gates that are not 0 is one, however many: also where the gates' product
    is below the type's range.  Through a gate of 0 it becomes NaN."""
    g = torch.Generator().manual_seed(T)
    x = torch.randn(1, T, D, generator=g)
    la = la0 * (0.75 + 0.25 * torch.rand(1, T, D, generator=g))
    dout = torch.randn(1, T, D, generator=g)
    x[0, 10, 0], x[0, 3, 1], dout[0, T - 5, 0], dout[0, T - 2, 1] = float("inf"), -float("inf"), float("inf"), -float("inf")
    la[0, T // 2, 1] = -float("inf")
    cu = [0, T // 3, T // 3, T - 1] if packed else None
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32).cuda()
    xd, ld, dd = dev(x, la, dout)
    out = LL.loglinear_glr_fwd(xd, ld, cu_seqlens=c, scale="one_minus")
    dx, dla, _ = LL.loglinear_glr_bwd(xd, ld, out, dd, cu_seqlens=c, scale="one_minus")
    n = T if cu is None else cu[-1]
    with np.errstate(invalid="ignore"):
        want, _ = oracle.glr_forward(x, la, "one_minus", cu=cu)
        grads = oracle.glr_backward(x, la, out, dout, "one_minus", cu=cu)
    for got, w, name in ((out, want, "out"), (dx, grads[0], "dx"), (dla, grads[1], "dlog_a")):
        got, w = to64(got)[:, :n], w[:, :n]
        fin = np.isfinite(w)
        assert np.array_equal(got[~fin], w[~fin], equal_nan=True), name
        check(torch.from_numpy(got[fin]).float(), w[fin], name)
    assert np.isinf(want[0, T // 3 - 1, 0]) and np.isinf(to64(dx)[0, 2 * T // 3, 0])


def test_gradients_behind_the_last_sequence_stay(LL):
    """Results that are given: rows that no sequence has are left as they are."""
    T, D, cu = 200, 12, [0, 30, 77]
    x, la = make(1, T, D, seed=2)
    g = torch.Generator().manual_seed(1)
    h0, ds = torch.randn(2, D, generator=g), torch.randn(2, D, generator=g)
    dout = torch.randn(1, T, D, generator=g)
    for t in (x, la, dout):
        t[:, 77:] = float("nan")
    xd, ld, hd, sd, dd = dev(x, la, h0, ds, dout)
    c = torch.tensor(cu, dtype=torch.int32).cuda()
    out = LL.loglinear_glr_fwd(xd, ld, h0=hd, cu_seqlens=c, scale="sqrt")
    dx, dla = torch.zeros(1, T, D).cuda(), torch.zeros(1, T, D).cuda()
    got = LL.loglinear_glr_bwd(xd, ld, out, dd, h0=hd, cu_seqlens=c, scale="sqrt", dstate=sd, dx=dx, dlog_a=dla, dh0=sd)
    assert got[0] is dx and got[1] is dla and got[2] is sd
    assert torch.all(dx[:, 77:] == 0) and torch.all(dla[:, 77:] == 0)
    want = oracle.glr_backward(x[:, :77], la[:, :77], out[:, :77], dout[:, :77], "sqrt", h0=h0, dstate=ds, cu=cu)
    for a, b in zip((dx[:, :77], dla[:, :77], sd), want):
        check(a.cpu(), b)


@pytest.mark.parametrize("cu", [None, [0, 0, 5, 300, 300, 1700, 1990, 1990]])
def test_state_gradients_in_place(LL, cu):
    """dstate and dh0 may be one array, empty sequences included; and packed states in place."""
    import ctypes
    from log_linear_attention_fwd_gb300 import _binding
    B, T, D = (2, 2000, 70) if cu is None else (1, 2000, 70)
    n = B if cu is None else len(cu) - 1
    x, la = dev(*make(B, T, D, seed=3))
    g = torch.Generator().manual_seed(1)
    h0, ds, dout = (torch.randn(*s, generator=g).cuda() for s in ((n, D), (n, D), (B, T, D)))
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32).cuda()
    state, both = torch.empty_like(h0), h0.clone()
    out = LL.loglinear_glr_fwd(x, la, h0=h0, state=state, scale="sqrt", cu_seqlens=c)
    again = LL.loglinear_glr_fwd(x, la, h0=both, state=both, scale="sqrt", cu_seqlens=c)
    end = T if cu is None else cu[-1]
    assert torch.equal(out[:, :end], again[:, :end]) and torch.equal(state, both)
    want = LL.loglinear_glr_bwd(x, la, out, dout, h0=h0, dstate=ds, scale="sqrt", cu_seqlens=c)
    both, dx, dla = ds.clone(), torch.empty_like(x), torch.empty_like(la)
    p = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())  # noqa: E731
    st = _binding.lib().loglinear_glr_bwd(p(x), None, p(la), None, p(h0), p(c), n, p(out), p(dout), p(both), p(dx),
                                          p(dla), p(both), B, T, D, 0, 0, 0, 2,
                                          ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0
    assert all(torch.equal(a[:, :end], b[:, :end]) for a, b in zip((dx, dla), want)) and torch.equal(both, want[2])


@pytest.mark.parametrize("scale", ["none", "one_minus", "sqrt"])
@pytest.mark.parametrize("dtype,gate", [("f32", "f32"), ("bf16", "bf16")])
def test_step_scales(LL, scale, dtype, gate):
    B, T, D = 2, 5, 33
    x, la = make(B, T, D, dtype, gate, seed=4)
    h0 = torch.randn(B, D, generator=torch.Generator().manual_seed(1))
    want, last = oracle.glr_forward(x, la, scale, h0=h0)
    state = h0.cuda()
    for t in range(T):
        check(LL.loglinear_glr_step(state, x[:, t].contiguous().cuda(), la[:, t].contiguous().cuda(), scale=scale).cpu(),
              want[:, t])
    check(state.cpu(), last)
