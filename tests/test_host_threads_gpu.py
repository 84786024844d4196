"""Calls from several host threads at once, whose shared memory differs while their kernel is the same: each
is served, with the results of calls one after the other."""
import threading

import pytest
import torch

import workloads as W
from tests.test_cache_gpu import i32, same, snapshot
from tests.test_tree_gpu import contexts, parents_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def LL():
    import log_linear_attention_fwd_gb300 as m
    return m


def recorded(monkeypatch, call):
    """The library calls that `call` makes, which it makes once: (function, arguments), the last one the stream."""
    from log_linear_attention_fwd_gb300 import _binding
    made, real = [], _binding._lib

    class Recorder:
        def __getattr__(self, name):
            fn = getattr(real, name)

            def record(*args):
                made.append((fn, args))
                return fn(*args)
            return fn if name.endswith("_size") else record

    with monkeypatch.context() as m:
        m.setattr(_binding, "_lib", Recorder())
        call()
    return made


def at_once(works, times):
    """Makes each work's calls in a host thread of its own, on a stream of its own, `times` times."""
    failed, start, device = [], threading.Barrier(len(works)), torch.cuda.current_device()

    def run(calls, stream):
        torch.cuda.set_device(device)
        calls = [(fn, (*args[:-1], stream.cuda_stream)) for fn, args in calls]
        start.wait()
        for _ in range(times):
            for fn, args in calls:
                status = fn(*args)
                if status or failed:
                    failed.append((fn.__name__, status))
                    return

    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in works]
    threads = [threading.Thread(target=run, args=w) for w in zip(works, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_trees(LL, monkeypatch, dtype):
    works, outs, want = [], [], []
    for N, dk, dv, M in ((64, 128, 128, 12), (33, 16, 4, 2), (47, 64, 32, 5)):
        cache, slots, ctx, tree, x = contexts(LL, [70, 130], N, 2, 1, dk, dv, dtype, True, M=M)
        args = (cache, i32(slots), i32([70, 130]), i32(parents_of(2, N, "chain")), x["q"], x["k"], x["v"], x["log_a"], x["lam"])
        out = torch.zeros(2, N, 2, dv).cuda()
        works.append(recorded(monkeypatch, lambda: LL.loglinear_cache_tree(*args, out=out)))
        outs.append((out, args))
        want.append(out.clone())
    at_once(works, 20000)
    assert all(torch.equal(a, b) for (a, _), b in zip(outs, want))


def test_accepts(LL, monkeypatch):
    works, caches, want = [], [], []
    for dk, dv in ((128, 128), (16, 4), (64, 100)):
        cache, slots, ctx, tree, x = contexts(LL, [61, 125], 6, 2, 1, dk, dv, "f32", True)
        args = (cache, i32(slots), i32([61, 125]), i32([[0, 1, 2], [1, 2, 3]]), x["k"], x["v"], x["log_a"])
        new = i32([0, 0])
        works.append(recorded(monkeypatch, lambda: LL.loglinear_cache_accept(*args, new_pos=new)))
        assert new.tolist() == [64, 128]
        caches.append((cache, args, new))
        want.append(snapshot(cache))
    at_once(works, 20000)
    assert all(same(snapshot(c), w) and c.error() == 0 for (c, _, _), w in zip(caches, want))


@pytest.mark.parametrize("call", ["forward", "prefill", "backward", "delta forward", "step"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_other_calls(LL, monkeypatch, dtype, call):
    works, outs, want = [], [], []
    for T, chunk, dk, dv, L in ((70, 64, 128, 128, 12), (40, 16, 16, 4, 9), (65, 32, 64, 96, 10)):
        x = W.make_fwd_inputs(W.FwdConfig("c", 1, 2, T, dk, dv, chunk, L, dtype, True, "softplus", seed=T))
        x = {k: v.cuda() for k, v in x.items()}
        args = (x["q"], x["k"], x["v"], x["log_a"], x["lam"])
        ws = torch.zeros(1 << 24, dtype=torch.uint8).cuda()
        out, keep = torch.zeros_like(x["v"]), []
        if call == "forward":
            work = lambda: keep.append(LL.loglinear_fwd(*args, chunk, out=out, workspace=ws, path="simt"))  # noqa: E731
        elif call == "prefill":
            state = torch.zeros(1, 2, L, dk, dv).cuda()
            work = lambda: keep.extend(LL.loglinear_prefill(*args, chunk, out=out, state=state, workspace=ws, path="simt"))  # noqa: E731
        elif call == "backward":
            work = lambda: keep.extend(LL.loglinear_bwd(*args, x["v"], workspace=ws, path="simt"))  # noqa: E731
        elif call == "delta forward":
            k = torch.nn.functional.normalize(x["k"].float(), dim=-1).to(x["k"].dtype)
            args = (x["q"], k, x["v"], x["log_a"], torch.rand(1, T, 2).cuda(), x["lam"])
            work = lambda: keep.append(LL.loglinear_gdn_fwd(*args, out=out))  # noqa: E731
        else:
            cache, slots, ctx, tree, y = contexts(LL, [70, 130], 1, 2, 1, dk, dv, dtype, True)
            one = [None if y[n] is None else y[n][:, 0].contiguous() for n in ("q", "k", "v", "log_a", "lam")]
            at = (cache, i32(slots), i32([70, 130]))
            out = torch.zeros_like(one[2])
            work = lambda: keep.extend((LL.loglinear_cache_step(*at, *one, out=out), one, at))  # noqa: E731
        works.append(recorded(monkeypatch, work))
        outs.append((keep, args, ws, out))
        want.append([t.clone() for t in keep if torch.is_tensor(t)])
    at_once(works, 5000)
    for (keep, *_), w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip([t for t in keep if torch.is_tensor(t)], w))
