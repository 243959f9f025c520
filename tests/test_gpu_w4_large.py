"""The operators on 4-bit weights where offsets pass 32 bits: the last rows of a large product against a call on those rows alone,
the last experts of weights of more than 2^32 bytes against the same experts by themselves."""

import pytest
import torch

from nvfp4_block_scaled_quant_gb300 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def room():
    free, _ = torch.cuda.mem_get_info()
    if free < 100 << 30:
        pytest.skip("needs 100 GB of device memory")
    yield
    torch.cuda.empty_cache()


def codes(*shape, seed):
    return torch.randint(256, shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV, dtype=torch.uint8)


def scales(*shape, seed):
    return torch.rand(shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).bfloat16() * 0.01


def same(y, z):
    """Equal but for the order of the sums, which differs between kernels and splits: a step of bf16, and fp32 noise."""
    y, z = y.double(), z.double()
    assert ((y - z).abs() <= 2.0 ** -7 * z.abs() + 1e-3).all()


def test_linear_with_many_rows():
    M, K, N, tail = 600_000, 4096, 64, 512  # 2.46e9 elements of x
    x = torch.empty(M, K, dtype=torch.bfloat16, device=DEV).normal_(generator=torch.Generator(device=DEV).manual_seed(1))
    w = ops.w4_prepare(codes(N, K // 2, seed=2), scales(N, K // 128, seed=3))
    y = ops.w4_linear(x, w)
    same(y[-tail:], ops.w4_linear(x[-tail:], w))
    del x, y
    x = torch.empty(M, 64, dtype=torch.bfloat16, device=DEV).normal_(generator=torch.Generator(device=DEV).manual_seed(4))
    w = ops.w4_prepare(codes(4096, 32, seed=5), scales(4096, 1, seed=6))
    y = ops.w4_linear(x, w)  # 2.46e9 elements of y
    same(y[-tail:], ops.w4_linear(x[-tail:], w))
    assert ops.device_error() == (0, 0)


@pytest.mark.parametrize("M", [3, 40, 1000])
def test_linear_with_many_features(M):
    K, N = 8192, 600_000  # 2.46e9 bytes of codes, 4.9e9 elements where they are written out
    c, s = codes(N, K // 2, seed=7), scales(N, K // 128, seed=8)
    w = ops.w4_prepare(c, s)
    x = torch.randn(M, K, generator=torch.Generator(device=DEV).manual_seed(9), device=DEV).bfloat16()
    y = ops.w4_linear(x, w)
    first = N - N % 128 - 1024  # whole tiles before the tail
    small = ops.w4_prepare(c[first:].contiguous(), s[first:].contiguous())
    same(y[:, first:], ops.w4_linear(x, small))
    assert ops.device_error() == (0, 0)


def test_experts_of_more_than_4_gib():
    E, H, I, T = 330, 7168, 2048, 5
    c13, s13 = codes(E, 2 * I, H // 2, seed=10), scales(E, 2 * I, H // 128, seed=11)
    c2, s2 = codes(E, H, I // 2, seed=12), scales(E, H, I // 128, seed=13)
    w13, w2 = ops.w4_prepare(c13, s13, gated=True), ops.w4_prepare(c2, s2)
    assert w2.data.numel() < 2 ** 32 < w13.data.numel()
    g = torch.Generator(device=DEV).manual_seed(14)
    x = torch.randn(T, H, generator=g, device=DEV).bfloat16() * 0.1
    router = torch.randn(E, H, generator=g, device=DEV).bfloat16() * 0.01
    last = E - 6
    router[last:] = (x.float().mean(0) * 40 + torch.randn(6, H, generator=g, device=DEV) * 0.02).bfloat16()
    x = (x.float() + x.float().mean(0) * 3).bfloat16()
    assert (torch.topk(x.float() @ router.float().T, 4, dim=1).indices >= last).all()
    y = ops.w4_moe(x, router, w13, w2, 4)
    few13 = ops.w4_prepare(c13[last:].contiguous(), s13[last:].contiguous(), gated=True)
    few2 = ops.w4_prepare(c2[last:].contiguous(), s2[last:].contiguous())
    same(y, ops.w4_moe(x, router[last:].contiguous(), few13, few2, 4))  # the logits' sums have other splits
    assert ops.device_error() == (0, 0)


def test_norm_with_many_rows():
    M, K, tail = 300_000, 8192, 4096
    f = torch.empty(M, K, dtype=torch.bfloat16, device=DEV).normal_(generator=torch.Generator(device=DEV).manual_seed(15))
    g = torch.ones(K, dtype=torch.bfloat16, device=DEV)
    r_out, q, s, y = ops.residual_norm_fp8(f, f, g, want_y=True)
    r2, q2, s2, y2 = ops.residual_norm_fp8(f[-tail:], f[-tail:], g, want_y=True)
    assert torch.equal(r_out[-tail:], r2) and torch.equal(y[-tail:], y2)
    assert torch.equal(q[-tail:].view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s[:, -tail:], s2)
    assert ops.device_error() == (0, 0)
