"""Calls of the experts' products that their documentation allows and whose
faults depend on timing, on other calls or on unusual values, against the
bounds of test_gpu_experts."""
import ctypes
import os
import subprocess
import sys
import threading

import pytest
import torch

import means_clustering_gmm_b200 as gmm
from means_clustering_gmm_b200 import _lib

from .test_gpu_experts import (DT, act, backward, check, cuda, dact, forward, half_step, inputs, tiny,
                               workspace)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("h,gated", [(0, False), (600, True)])
def test_biases_of_the_next_tile(h, gated):
    """Blocks that work through many tiles, experts and columns whose biases
    are far apart, and tiles of which some rows hold no point: a bias read
    from the tile after would be off by whole numbers."""
    N, d, o, K = 9000, 64, 1104, 5
    s = inputs(41, N, d, h, o, K, 1, "f16", gated=gated, cut=0.2, use=[0, 0, 0, 1, 3, 4])
    step = torch.arange(s["b1"].shape[1]) // 32 % 7
    s["b1"] = (s["b1"] + torch.arange(K)[:, None] - step).half()
    check(s, "silu", gated)


def routed(seed, N, d, h, o, K, r, dtype="bf16"):
    c = {k: t.cuda() if isinstance(t, torch.Tensor) else t
         for k, t in inputs(seed, N, d, h, o, K, r, dtype).items()}
    return c, workspace(c, False, False)


@pytest.mark.parametrize("sizes", [
    [dict(N=64, K=9, r=4), dict(N=1, K=9, r=4)],          # few points
    [dict(N=100, K=300, r=2), dict(N=100, K=1000, r=2)],  # one-block routing
    [dict(N=100, K=3100, r=2), dict(N=100, K=4096, r=2)],     # routing in steps
])
def test_threads_with_calls_of_different_sizes(sizes):
    """Host threads, each with its stream and workspace, whose calls need
    different amounts of shared memory of the same kernels."""
    lib = _lib.load()
    failed, results = [], []

    def loop(c, ws, stream, y):
        s = c["x"].shape + c["w2"].shape + c["ids"].shape
        shape = _lib.ExpertShape(N=s[0], d=s[1], h=s[4], o=s[3], K=s[2], r=s[6],
                                 dtype=_lib.GMM_BF16, activation=3, gated=0)
        args = [ctypes.byref(shape)] + [
            ctypes.c_void_p(c[k].data_ptr()) for k in ("x", "ids", "resp", "w1", "b1", "w2", "b2")]
        args += [None, ctypes.c_void_p(y.data_ptr()), ctypes.c_void_p(ws.ptr), ws.nbytes, 0,
                 ctypes.c_void_p(stream.cuda_stream)]
        for i in range(10000):
            status = lib.gmm_expert_mlp(*args)
            if status:
                failed.append(status)
            if i % 100 == 99:
                stream.synchronize()

    threads = []
    for i, kw in enumerate(2 * sizes):
        c, ws = routed(50 + i, d=64, h=64, o=64, **kw)
        want = forward(c, "silu", ws=ws)[0]
        results.append((torch.empty_like(want), want))
        args = (c, ws, torch.cuda.Stream(), results[-1][0])
        threads.append(threading.Thread(target=loop, args=args))
    torch.cuda.synchronize()
    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    torch.cuda.synchronize()
    assert not failed, (len(failed), set(failed))
    assert all(torch.equal(got, want) for got, want in results)


FIRST_CALLS = """
import threading, torch
import means_clustering_gmm_b200 as gmm
def call():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(2000, 64, generator=g).bfloat16().cuda()
    w = torch.randn(1, 128, 64, generator=g).bfloat16().cuda()
    ws = gmm.Workspace.for_expert_linear(2000, 64, 128, 1, 0, x.dtype, backward=True)
    barrier.wait()
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda.current_stream().wait_stream(torch.cuda.default_stream())
        y = gmm.expert_linear(x, None, None, w, None, ws, "silu")
        got = gmm.expert_linear_backward(y, x, None, None, w, None, ws, "silu")[:2] + (y,)
    torch.cuda.synchronize()
    results.append(got)
results, barrier = [], threading.Barrier(6)
threads = [threading.Thread(target=call) for _ in range(6)]
[t.start() for t in threads]
[t.join() for t in threads]
assert len(results) == 6
assert all(torch.equal(a, b) for r in results for a, b in zip(r, results[0]))
print("equal")
"""


def test_first_calls_on_several_threads():
    """The first calls of a process, made at once: what the library asks the
    device for once is asked by several threads."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True,
                         text=True, timeout=120)
    assert run.returncode == 0 and "equal" in run.stdout, run.stderr[-2000:]


def test_gradient_over_a_billion_points():
    """A weight gradient whose contraction, one tile's, takes longer than the
    limit of an ordinary wait."""
    N, d, o = 1_400_000_000, 8, 8
    rows = [0, 63, 64, N // 2, 2 ** 30 + 1, N - 65, N - 1]
    g = torch.Generator().manual_seed(61)
    some = torch.randint(-3, 4, (2, len(rows), d), generator=g).bfloat16()
    x = torch.zeros(N, d, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros(N, o, dtype=torch.bfloat16, device="cuda")
    x[rows], dy[rows] = some[0].cuda(), some[1].cuda()
    w = torch.eye(8, dtype=torch.bfloat16, device="cuda")[None]
    ws = gmm.Workspace.for_expert_linear(N, d, o, 1, 0, x.dtype, backward=True)
    dX, dW, _, _ = gmm.expert_linear_backward(dy, x, None, None, w, None, ws)
    assert gmm.gmm_last_error(ws) == 0
    assert torch.equal(dW[0].cpu().float(), some[1].float().T @ some[0].float())
    assert torch.equal(dX[rows].cpu(), some[1]) and not dX[1:63].any()


@pytest.mark.parametrize("flags", [0, gmm.GMM_FLAG_FORCE_SIMT])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("N,d,h,o,r", [(40, 7, 5, 3, 2), (70, 8, 13, 8, 1), (900, 50, 61, 70, 1),
                                       (90, 64, 72, 64, 2)])
def test_an_infinity_behind_relu(N, d, h, o, r, dtype, flags):
    """Hidden units at minus infinity are 0 behind relu, and so is their
    gradient: a point with an infinite coordinate has the results of one with a
    large coordinate, whatever copies the widths need.  Only dW1 of its experts
    holds 0 * inf, in that coordinate's column."""
    s = inputs(71, N, d, h, o, 3, r, dtype)
    s["w1"][:, :, 2] = -s["w1"][:, :, 2].abs() - 1
    big = dict(s, x=s["x"].clone())
    big["x"][5, 2] = 2.0 ** 14
    inf = dict(s, x=s["x"].clone())
    inf["x"][5, 2] = float("inf")
    y, want = (forward(cuda(t), "relu", flags=flags)[0] for t in (inf, big))
    assert want.isfinite().all() and torch.equal(y, want)
    got, want = (backward(cuda(t), "relu", flags=flags)[0] for t in (inf, big))
    for t in (got, want):
        t["dw1"][s["ids"][5].long(), :, 2] = 0
    for k in want:
        assert want[k].isfinite().all() and torch.equal(got[k], want[k]), k


@pytest.mark.parametrize("h", [0, 72])
def test_arrays_may_be_dropped_after_a_call_on_a_stream(h):
    """What a call with ``stream`` still has to read is not handed out again:
    the stream is kept busy, everything dropped, and new arrays of the same
    sizes get other memory."""
    c = cuda(inputs(81, 300, 64, h, 64, 3, 2, "bf16", res=True))
    want, want_g = forward(c, "silu")[0], backward(c, "silu")[0]
    side = torch.cuda.Stream()
    for call, keep in ((forward, ("w1", "w2", "b1", "b2", "x", "ids", "resp", "res")),
                       (backward, ("w1", "w2", "b1", "b2", "x", "ids", "resp", "dy"))):
        call(c, "silu", stream=side)   # (the stream's own memory)
        s = {k: t.clone() if isinstance(t, torch.Tensor) else t for k, t in c.items()}
        ws = workspace(s, False, call is backward)
        torch.cuda.synchronize()
        busy = {t.data_ptr(): (t.shape, t.dtype) for t in
                [s[k] for k in keep if s[k] is not None] + [ws.buf]}
        with torch.cuda.stream(side):
            torch.cuda._sleep(1_000_000_000)   # clocks: 0.5 s
        got = call(s, "silu", ws=ws, stream=side)[0]
        del s, ws
        new = [torch.empty(v[0], dtype=v[1], device="cuda") for v in busy.values()]
        assert not side.query()   # (otherwise nothing is shown)
        assert not busy.keys() & {t.data_ptr() for t in new}
        for t in new:
            t.fill_(1)
        torch.cuda.synchronize()
        if call is forward:
            assert torch.equal(got, want)
        else:
            assert all(torch.equal(got[k], want_g[k]) for k in want_g)


@pytest.mark.parametrize("N", [64, 1600])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("activation", ["gelu", "silu"])
def test_activations_of_16_bit_calls(activation, dtype, N):
    """f and f' at known arguments (identity weights), as include/gmm_b200.h
    bounds them.  gelu: 2^-23 of |z| from the distribution function (its
    formula's 7.5e-8 is 2^-23.7, its fp32 sums the rest), and the exponential's
    2^-20 (1 + z^2) relative to the tail.  silu: relative to f, 2^-20 + |z| 2^-23.
    Results are rounded once, the gradient twice (da is rounded too)."""
    dt, n8 = DT[dtype], N * 8
    z = torch.cat([torch.linspace(-14, 14, n8 - 8), torch.tensor([0.0, -0.0, 60, -60, 80, -80, 200,
                                                                  -200])]).to(dt).view(N, 8)
    one = torch.ones(N, 8, dtype=dt)
    w = torch.eye(8, dtype=dt)[None].cuda()
    ws = gmm.Workspace.for_expert_linear(N, 8, 8, 1, 0, dt, backward=True)
    y = gmm.expert_linear(z.cuda(), None, None, w, None, ws, activation).cpu().double()
    dx = gmm.expert_linear_backward(one.cuda(), z.cuda(), None, None, w, None, ws,
                                    activation)[0].cpu().double()
    z = z.double()
    f, df = act(z, activation), dact(z, activation)
    if activation == "gelu":
        tail = 0.5 * torch.erfc(z.abs() / 2 ** 0.5)
        cdf = 2.0 ** -23 + 2.0 ** -20 * (1 + z * z) * tail
        ef = z.abs() * cdf
        edf = cdf + (2.0 ** -20 + 2.0 ** -22 * z * z) * z.abs() * torch.exp(-z * z / 2)
    else:
        rel = 2.0 ** -20 + 2.0 ** -23 * z.abs()
        p = torch.sigmoid(z)
        ef = rel * f.abs() + 2.0 ** -126 * z.abs()
        edf = rel * (p + 2 * f.abs()) + 2.0 ** -126 * (1 + z.abs())
    u = half_step(dt)
    assert ((y - f).abs() <= ef + u * (f.abs() + ef) + tiny(dt)).all()
    err = (dx - df).abs() - (edf + 2 * u * (1 + u) * (df.abs() + edf) + 2 * tiny(dt))
    assert (err <= 0).all(), (err.max(), z.flatten()[err.argmax()])


@pytest.mark.parametrize("N,d,o,dtype", [(3, 64, 72, "bf16"), (300, 64, 72, "f16"),
                                         (300, 33, 21, "bf16"), (40, 64, 24, "f32")])
def test_a_captured_fork_and_join(N, d, o, dtype):
    """Inside one graph: inputs written on one stream just before calls on it
    and on another one, a workspace each, both joined and their results added;
    replayed with new contents."""
    c = cuda(inputs(91, N, d, 48, o, 5, 2, dtype, res=True, cut=0.2))
    spaces = [workspace(c, False, True) for _ in range(2)]
    fresh = {k: c[k].clone() for k in ("x", "dy", "resp", "ids")}
    side = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        for k, t in fresh.items():
            c[k].copy_(t)
        side.wait_stream(here)
        y = forward(c, "silu", ws=spaces[0])[0]
        with torch.cuda.stream(side):
            g = backward(c, "silu", ws=spaces[1])[0]
            g["dx"].mul_(2)
        here.wait_stream(side)
        return forward(dict(c, res=y), "silu", ws=spaces[1])[0], g

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, g = step()
    for turn in range(3):
        fresh["x"].copy_(torch.randn(N, d, device="cuda"))
        fresh["ids"].copy_(torch.randint(-1, 5, (N, 2), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        want_y, want_g = step()
        torch.cuda.synchronize()
        assert torch.equal(y, want_y) and all(torch.equal(g[k], want_g[k]) for k in want_g)


@pytest.mark.parametrize("N,r,h", [(5, 2, 0), (300, 1, 0), (300, 2, 31), (300, 0, 31), (900, 1, 30)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_result_may_replace_the_residual_at_odd_widths(N, r, h, dtype):
    c = cuda(inputs(92, N, 33, h, 21, 3 if r else 1, r, dtype, res=True))
    want = forward(c, "silu")[0]
    assert torch.equal(forward(c, "silu", out=c["res"])[0], want)


@pytest.mark.parametrize("K,N,r", [(4096, 700, 8), (4096, 20, 8), (1023, 2000, 2), (1024, 500, 1)])
@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_many_experts(K, N, r, dtype):
    """The most experts, and both sides of the one-block routing's limit."""
    check(inputs(93, N, 16, 0, 8, K, r, dtype, cut=0.1), "silu")


@pytest.mark.parametrize("N,d,h,o,r,dtype,flags", [
    (300, 33, 21, 65, 2, "bf16", 0), (40, 31, 0, 27, 1, "f16", 0), (3, 33, 40, 65, 2, "bf16", 0),
    (700, 64, 61, 50, 1, "f16", 0), (300, 33, 21, 65, 2, "f32", 0), (20, 30, 0, 26, 1, "f32", 0),
    (300, 64, 0, 27, 0, "f32", 0), (300, 33, 21, 65, 2, "bf16", gmm.GMM_FLAG_FORCE_SIMT),
    (300, 50, 0, 64, 2, "f16", gmm.GMM_FLAG_FORCE_SIMT)])
def test_odd_widths_at_any_element(N, d, h, o, r, dtype, flags):
    """Arrays whose rows are not whole 16-byte units may start at any element
    (slices of rows do), the others at 16 bytes."""
    s = inputs(95, N, d, h, o, 4 if r else 1, r, dtype, res=True)
    want = forward(cuda(s), "silu", flags=flags)[0], backward(cuda(s), "silu", flags=flags)[0]
    size = s["x"].element_size()

    def shifted(t, k=1):
        k = k if t.shape[-1] * size % 16 else 16 // size
        room = torch.empty(t.numel() + k, dtype=t.dtype, device="cuda")
        return room[k:].view(t.shape).copy_(t)

    c = {k: shifted(t) if isinstance(t, torch.Tensor) and k not in ("ids", "resp") else
         t.cuda() if isinstance(t, torch.Tensor) else t for k, t in s.items()}
    out = shifted(torch.zeros(N, o, dtype=DT[dtype]), 3)
    assert torch.equal(forward(c, "silu", flags=flags, out=out)[0], want[0])
    got = backward(c, "silu", flags=flags)[0]
    assert all(torch.equal(got[k], want[1][k]) for k in want[1])
