"""Launches of kernels on CTA pairs run one after the other on a device, on whatever streams they are
queued: a short one queued behind a long one on another stream ends after it, and so do the branches
of a captured graph.  The results are those of the calls by themselves."""

import ctypes
import threading

import pytest
import torch

from nvfp4_block_scaled_quant_gb300 import _lib, model, ops

pytestmark = pytest.mark.gpu
DEV = "cuda"


def fp8(M, K, N, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = ops.fp8_quantize_act(torch.randn(M, K, generator=g, device=DEV).bfloat16())
    w = ops.fp8_quantize_weight(torch.randn(N, K, generator=g, device=DEV).bfloat16())
    return lambda: ops.fp8_gemm(*x, *w)


def gated(T, H, I, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x, dh = (torch.randn(T, n, generator=g, device=DEV).bfloat16() for n in (H, I))
    wg, wu = ((torch.randn(I, H, generator=g, device=DEV) * H ** -0.5).bfloat16() for _ in range(2))

    def step():
        _, gu = ops.gated_linear(x, wg, wu, save=True)
        return ops.gated_linear_backward(dh, x, wg, wu, gu)[0]

    return step


def nvfp4(M, K, N, seed):
    w = model.make_dense_weight(N, K, seed=seed, device=DEV)
    x = torch.randn(M, K, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).bfloat16()
    return lambda: ops.linear(x, w.w, w.sf, w.ws2, N)[0]


SHORT = {"fp8": lambda: fp8(300, 256, 256, 1), "gated": lambda: gated(300, 128, 128, 2), "nvfp4": lambda: nvfp4(2048, 256, 256, 3)}


@pytest.mark.parametrize("kind", list(SHORT))
def test_a_short_launch_on_another_stream_ends_after_the_long_one(kind):
    long, short = fp8(4096, 7168, 7168, 4), SHORT[kind]()
    want_long, want_short = long(), short()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for first, second in ((a, b), (b, a)):
        ends = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
        with torch.cuda.stream(first):
            got = [long()]
            ends[0].record()
        with torch.cuda.stream(second):
            got.append(short())
            ends[1].record()
        with torch.cuda.stream(first):
            got.append(long())
            ends[2].record()
        torch.cuda.synchronize()
        assert ends[0].elapsed_time(ends[1]) > 0 and ends[1].elapsed_time(ends[2]) > 0
        assert torch.equal(got[0], want_long) and torch.equal(got[1], want_short) and torch.equal(got[2], want_long)
    assert ops.device_error() == (0, 0)


def test_products_of_different_grids_in_turn():
    """NVFP4 and FP8 products on CTA pairs with different numbers of pairs, queued without waiting, also in a graph."""
    calls = [nvfp4(2048, 512, 1024, 7), fp8(900, 384, 520, 8), nvfp4(600, 768, 512, 9), gated(700, 264, 520, 10)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    got = [[c() for c in calls] for _ in range(5)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = [c() for _ in range(2) for c in calls]
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for g in [*got, held[:4], held[4:]]:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
    assert ops.device_error() == (0, 0)


@pytest.mark.parametrize("kind", list(SHORT))
def test_branches_of_a_captured_graph(kind):
    long, short = fp8(4096, 7168, 7168, 5), SHORT[kind]()
    want = long(), short()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    ends = [torch.cuda.Event(enable_timing=True, external=True) for _ in range(2)]
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        x = long()
        ends[0].record()
        with torch.cuda.stream(side):
            y = short()
            ends[1].record()
        here.wait_stream(side)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert ends[0].elapsed_time(ends[1]) > 0
    with torch.cuda.stream(side):  # what a capture recorded orders nothing outside it
        eager = short()
    torch.cuda.synchronize()
    assert torch.equal(x, want[0]) and torch.equal(y, want[1]) and torch.equal(eager, want[1])
    assert ops.device_error() == (0, 0)


def test_captures_at_the_same_time_keep_their_own_order():
    """Two captures go on at once; the second branch of the first one still starts behind its first branch's product,
    whatever the other capture recorded in between."""
    rt = ctypes.CDLL("libcudart.so." + torch.version.cuda.split(".")[0])
    M, K, N = 600, 256, 512
    x, xs = ops.fp8_quantize_act(torch.ones(M, K, dtype=torch.bfloat16, device=DEV))
    w, ws = ops.fp8_quantize_weight(torch.ones(N, K, dtype=torch.bfloat16, device=DEV))
    y = [torch.empty(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(3)]

    def product(out, stream):
        _lib.call("nvfp4_fp8_gemm", x.data_ptr(), xs.data_ptr(), xs.stride(0), M, K, N, w.data_ptr(), ws.data_ptr(), _lib.DT_BF16,
                  out.data_ptr(), stream.cuda_stream)

    a, branch, b = (torch.cuda.Stream() for _ in range(3))
    for s in (a, branch, b):
        product(y[0], s)
    torch.cuda.synchronize()
    handles = [ctypes.c_void_p(s.cuda_stream) for s in (a, b)]
    for h in handles:
        assert rt.cudaStreamBeginCapture(h, 2) == 0  # relaxed
    fork, join = torch.cuda.Event(), torch.cuda.Event()
    fork.record(a)
    branch.wait_event(fork)
    product(y[0], a)
    product(y[1], b)
    product(y[2], branch)
    join.record(branch)
    a.wait_event(join)
    roots = []
    for h in handles:
        graph, n = ctypes.c_void_p(), ctypes.c_size_t()
        assert rt.cudaStreamEndCapture(h, ctypes.byref(graph)) == 0
        assert rt.cudaGraphGetRootNodes(graph, None, ctypes.byref(n)) == 0
        roots.append(n.value)
        assert rt.cudaGraphDestroy(graph) == 0
    assert roots == [1, 1]  # the branch's product is no root of its graph
    torch.cuda.synchronize()


def test_calls_from_several_threads():
    """Threads with a stream of their own: the launches of each are in its stream's order and in turn with the others'."""
    calls = [fp8(600, 512, 512, 20), gated(300, 256, 264, 21), nvfp4(1024, 256, 512, 22), fp8(40, 512, 512, 23)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    got = [None] * len(calls)

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            got[i] = [calls[i]() for _ in range(30)]
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for outs, w in zip(got, want):
        assert outs is not None and all(torch.equal(o, w) for o in outs)
    assert ops.device_error() == (0, 0)
