"""The linear layer on 4-bit weights with group scales, against its definition in 64 bits."""

import pytest
import torch

from nvfp4_block_scaled_quant_gb300 import ops
from w4_reference import F64, TYPES, check, checkpoint, product

pytestmark = pytest.mark.gpu


def make(M, K, N, group, zeros, kind, seed=0):
    g = torch.Generator(device="cuda").manual_seed(1000 * seed + M + K + N)
    dt = TYPES[kind]
    ck = checkpoint(g, (N, K), group, zeros, dt, "cuda")
    x = (torch.randn(M, K, generator=g, device="cuda") * torch.exp(0.7 * torch.randn(K, generator=g, device="cuda"))).to(dt)
    return x, ck, ops.w4_prepare(*ck, group=group)


def verify(x, ck, group, y, what=""):
    want, err = product(x.to(F64), ck, group)
    check(y, want, err, x.dtype, what)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("group,zeros", [(32, False), (32, True), (64, False), (64, True), (128, False), (128, True)])
@pytest.mark.parametrize("M,K,N", [(1, 128, 64), (3, 264, 65), (8, 1000, 200), (9, 2000, 137), (16, 512, 96), (17, 1544, 130),
                                   (64, 384, 256), (100, 904, 300), (300, 264, 140)])
def test_sizes(M, K, N, group, zeros, kind):
    x, ck, w = make(M, K, N, group, zeros, kind)
    verify(x, ck, group, ops.w4_linear(x, w))


@pytest.mark.parametrize("M,K,N", [(1, 8, 1), (1, 24, 3), (2, 136, 1), (5, 40, 63), (40, 8, 2), (1, 7168, 2048), (13, 1536, 16384),
                                   (33, 7168, 72), (129, 4104, 1), (257, 136, 513), (1, 16384, 24)])
def test_small_large_and_odd(M, K, N):
    x, ck, w = make(M, K, N, 64, True, "bf16", 1)
    verify(x, ck, 64, ops.w4_linear(x, w))


@pytest.mark.parametrize("M", [1, 12, 50, 200])
def test_strided_rows_and_out(M):
    x, ck, w = make(M, 520, 100, 128, False, "fp16", 2)
    wide = torch.full((M, 704), float("nan"), device="cuda", dtype=x.dtype)
    wide[:, 88:608] = x
    rows = wide[:, 88:608]
    out = torch.empty(M, 100, device="cuda", dtype=x.dtype)
    y = ops.w4_linear(rows, w, out=out)
    assert y is out
    assert torch.equal(y, ops.w4_linear(x, w))
    verify(x, ck, 128, y)


@pytest.mark.parametrize("M", [1, 16, 40, 300])
def test_rows_do_not_mix_and_repeat(M):
    x, _, w = make(M, 1032, 200, 32, True, "bf16", 3)
    y = ops.w4_linear(x, w)
    for _ in range(3):
        assert torch.equal(ops.w4_linear(x, w), y)
    bad = x.clone()
    bad[M - 1, 5] = float("inf")
    z = ops.w4_linear(bad, w)
    assert torch.equal(z[:M - 1], y[:M - 1])
    assert not torch.isfinite(z[M - 1]).any()


def test_no_rows():
    x, _, w = make(1, 64, 32, 32, False, "bf16", 4)
    assert ops.w4_linear(x[:0], w).shape == (0, 32)


@pytest.mark.parametrize("M", [1, 30, 150])
def test_extreme_codes_and_scales(M):
    """All codes and zero points at their ends, scales at the ends of fp16's range."""
    K, N, group = 256, 70, 128
    g = torch.Generator(device="cuda").manual_seed(5)
    codes = torch.randint(0, 2, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8) * 255
    zeros = torch.randint(0, 2, (N, 2), generator=g, device="cuda", dtype=torch.uint8) * 15
    scales = torch.tensor([6e-8, 1e-4, 1.0, 60000.0], device="cuda")[torch.randint(0, 4, (N, 2), generator=g, device="cuda")].half()
    x = (torch.randn(M, K, generator=g, device="cuda") * 1e-3).half()
    ck = (codes, scales, zeros)
    verify(x, ck, group, ops.w4_linear(x, ops.w4_prepare(*ck, group=group)))


def test_high_bits_of_zero_points_do_not_count():
    x, ck, w = make(4, 128, 40, 32, True, "bf16", 6)
    dirty = ops.w4_prepare(ck[0], ck[1], ck[2] | 0xA0, group=32)
    assert torch.equal(w.data, dirty.data)
    assert torch.equal(ops.w4_linear(x, w), ops.w4_linear(x, dirty))


@pytest.mark.parametrize("M", [2, 80])
def test_stream_and_graph(M):
    x, ck, w = make(M, 776, 333, 64, False, "bf16", 7)
    want = ops.w4_linear(x, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.w4_linear(x, w, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    static = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ops.w4_linear(static, w)
        z = ops.w4_linear(static, w)
    for k in range(3):
        static.copy_(torch.roll(x, k, 0))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, torch.roll(want, k, 0)) and torch.equal(z, y)


@pytest.mark.parametrize("group,zeros,kind", [(128, False, "bf16"), (128, True, "fp16"), (64, True, "bf16"), (32, False, "fp16"), (32, True, "bf16")])
@pytest.mark.parametrize("M,K,N", [(1100, 136, 1160), (900, 264, 2056), (2100, 776, 1137), (1281, 200, 4104), (600, 520, 4100), (3001, 264, 1048),
                                   (513, 64, 16392), (700, 72, 8200)])
def test_many_rows(M, K, N, group, zeros, kind):
    """Sizes that go through written-out weights: edges inside tiles of either direction, outputs of whole 16-byte rows and others, groups
    and K blocks that end early; nothing is written outside of y."""
    x, ck, w = make(M, K, N, group, zeros, kind, 8)
    pad = 4096
    flat = torch.full((M * N + 2 * pad,), 7.0, device="cuda", dtype=x.dtype)
    y = ops.w4_linear(x, w, out=flat[pad:pad + M * N].view(M, N))
    verify(x, ck, group, y)
    assert (flat[:pad] == 7).all() and (flat[pad + M * N:] == 7).all()
    assert torch.equal(ops.w4_linear(x, w), y)


def test_many_rows_do_not_mix():
    x, _, w = make(1500, 264, 1048, 128, False, "bf16", 9)
    y = ops.w4_linear(x, w)
    bad = x.clone()
    bad[700, 5] = float("nan")
    z = ops.w4_linear(bad, w)
    assert torch.equal(torch.cat([z[:700], z[701:]]), torch.cat([y[:700], y[701:]]))
    assert not torch.isfinite(z[700]).any()
