"""The operators on 4-bit weights with scales and activations at the ends of their range, against the definition in 64 bits."""

import pytest
import torch

from nvfp4_block_scaled_quant_gb300 import ops
from w4_reference import F64, check, checkpoint, moe, product, weight

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


@pytest.mark.parametrize("power", [-60, -76, -90, -110])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("M", [1, 5, 16, 40, 1100])
def test_small_bf16_scales(M, group, zeros, power):
    """Scales down to 2^-114: outputs are ordinary bf16 numbers, to the same bound as under scales around one."""
    g = torch.Generator(device=DEV).manual_seed(M + group)
    K, N = 520, 200
    ck = checkpoint(g, (N, K), group, zeros, BF, DEV)
    ck = (ck[0], (ck[1].float() * 2.0 ** power).to(BF), ck[2])
    x = torch.randn(M, K, generator=g, device=DEV).to(BF)
    want, err = product(x.to(F64), ck, group)
    check(ops.w4_linear(x, ops.w4_prepare(*ck, group=group)), want, err, BF)


@pytest.mark.parametrize("up,down", [(0, -80), (-60, -40), (-100, 0)])
@pytest.mark.parametrize("T", [1, 11])
def test_small_bf16_scales_of_experts(T, up, down):
    """The same for the up and the down projection of the experts."""
    g = torch.Generator(device=DEV).manual_seed(T)
    H, I, E, topk = 264, 136, 12, 3
    cks = []
    for shape, p in (((E, 2 * I, H), up), ((E, H, I), down), ((2 * I, H), up), ((H, I), down)):
        codes, scales, zeros = checkpoint(g, shape, 64, True, BF, DEV)
        power = torch.full(scales.shape, float(p), device=DEV)
        if shape[-1] == H:
            power[..., :I, :] = 0  # the gate keeps its size
        cks.append((codes, (scales.float() * torch.exp2(power)).to(BF), zeros))
    x = torch.randn(T, H, generator=g, device=DEV).to(BF)
    router = (torch.randn(E, H, generator=g, device=DEV) * H ** -0.5).to(BF)
    w13, w2, s13, s2 = (ops.w4_prepare(*c, group=64, gated=i % 2 == 0) for i, c in enumerate(cks))
    y = ops.w4_moe(x, router, w13, w2, topk, shared13=s13, shared2=s2)
    want, err, _, sure = moe(x.to(F64), router, cks[0], cks[1], topk, 64, "silu", BF, (cks[2], cks[3]))
    assert sure
    check(y, want, err, BF)


def without_column(ck, group, col):
    """The checkpoint with weights of zero (c = z) in one column."""
    codes, scales, zeros = (None if v is None else v.clone() for v in ck)
    z = torch.full_like(codes[..., col // 2], 8) if zeros is None else zeros[..., col // group]
    codes[..., col // 2] = codes[..., col // 2] & (0x0F if col % 2 else 0xF0) | z << (4 if col % 2 else 0)
    return codes, scales, zeros


OUTLIERS = [("bf16", 1e4, 1.0), ("bf16", 1e9, 1.0), ("bf16", 1e36, 1.0), ("fp16", 6e4, 1.0), ("fp16", 6e4, 2.0 ** -14), ("fp16", 6e4, 2.0 ** -20)]


@pytest.mark.parametrize("kind,outlier,size", OUTLIERS)
@pytest.mark.parametrize("group,zeros", [(32, False), (64, True), (128, False), (128, True)])
@pytest.mark.parametrize("M", [1, 7, 16, 40, 1100])
def test_outlier_that_meets_zero_weights(M, group, zeros, kind, outlier, size):
    """An activation that only meets weights of zero adds nothing: the bound is that of the row without it."""
    g = torch.Generator(device=DEV).manual_seed(M + group)
    dt, K, N, col = {"bf16": BF, "fp16": torch.float16}[kind], 392, 200, 131 if zeros else 134
    ck = without_column(checkpoint(g, (N, K), group, zeros, dt, DEV), group, col)
    # scales that bring the outputs of small rows into fp16's normal range
    ck = (ck[0], (ck[1].float() / max(size, 2.0 ** -14)).to(dt), ck[2])
    x = (torch.randn(M, K, generator=g, device=DEV) * size).to(dt)
    x[:, col] = 0
    want, err = product(x.to(F64), ck, group)
    x[:, col] = outlier
    check(ops.w4_linear(x, ops.w4_prepare(*ck, group=group)), want, err, dt)


@pytest.mark.parametrize("kind,outlier,size", OUTLIERS)
@pytest.mark.parametrize("group,zeros", [(32, True), (128, False)])
@pytest.mark.parametrize("T", [1, 13])
def test_outlier_that_meets_zero_weights_of_experts(T, group, zeros, kind, outlier, size):
    """The same in the experts' up projections, the router blind to the column too."""
    g = torch.Generator(device=DEV).manual_seed(T + group)
    dt, H, I, E, topk, col = {"bf16": BF, "fp16": torch.float16}[kind], 392, 136, 12, 3, 134
    cks = [checkpoint(g, s, group, zeros, dt, DEV) for s in ((E, 2 * I, H), (E, H, I), (2 * I, H), (H, I))]
    for i in (0, 2):
        codes, scales, z = without_column(cks[i], group, col)
        cks[i] = (codes, (scales.float() / max(size, 2.0 ** -14)).to(dt), z)
    x = (torch.randn(T, H, generator=g, device=DEV) * size).to(dt)
    router = (torch.randn(E, H, generator=g, device=DEV) * H ** -0.5).to(dt)
    router[:, col] = 0
    x[:, col] = 0
    want, err, _, sure = moe(x.to(F64), router, cks[0], cks[1], topk, group, "silu", dt, (cks[2], cks[3]))
    assert sure
    x[:, col] = outlier
    w13, w2, s13, s2 = (ops.w4_prepare(*c, group=group, gated=i % 2 == 0) for i, c in enumerate(cks))
    check(ops.w4_moe(x, router, w13, w2, topk, shared13=s13, shared2=s2), want, err, dt)


SIZES = (1.0, 300.0, 1e-2, 3000.0, 30.0, 1e4)


def wide_layer(T, H, I, E, topk, group, zeros, seed):
    """An fp16 layer whose hidden rows pass 65504 for some tokens while its outputs do not."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = torch.float16
    cks = [checkpoint(g, s, group, zeros, dt, DEV) for s in ((E, 2 * I, H), (E, H, I), (2 * I, H), (H, I))]
    for i in (1, 3):
        cks[i] = (cks[i][0], (cks[i][1].float() * 2.0 ** -10).to(dt), cks[i][2])
    x = torch.randn(T, H, generator=g, device=DEV) * torch.tensor(SIZES, device=DEV)[(torch.arange(T, device=DEV) + (T == 1)) % len(SIZES)][:, None]
    router = (torch.randn(E, H, generator=g, device=DEV) * H ** -0.5).to(dt)
    packed = [ops.w4_prepare(*c, group=group, gated=i % 2 == 0) for i, c in enumerate(cks)]

    def run(x):
        return ops.w4_moe(x, router, packed[0], packed[1], topk, shared13=packed[2], shared2=packed[3])

    return x.clamp(-6e4, 6e4).to(dt), router, cks, run


@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("T,H,I,E,topk", [(1, 264, 136, 8, 2), (6, 392, 40, 12, 3), (13, 64, 1000, 6, 2), (40, 136, 264, 5, 2), (64, 264, 72, 40, 8),
                                          (7, 8, 2056, 4, 2)])
def test_fp16_hidden_rows_past_the_range(T, H, I, E, topk, group, zeros):
    x, router, cks, run = wide_layer(T, H, I, E, topk, group, zeros, T + I)
    want, err, _, _ = moe(x.to(F64), router, cks[0], cks[1], topk, group, "silu", x.dtype, (cks[2], cks[3]))
    gu = x.to(F64) @ weight((cks[2][0], cks[2][1], cks[2][2]), group)[0].T
    assert (torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]).abs().max() > 65504  # of the shared expert
    fits = want.abs() + err < 65504
    assert fits.float().mean() > 0.5
    y = run(x)
    check(torch.where(fits, y, 0), torch.where(fits, want, 0), err, x.dtype)
    assert torch.equal(y, run(x))
    # the others' outputs do not hang on the large tokens
    keep = torch.arange(T, device=DEV) % len(SIZES) % 2 == 0
    if T > 1:
        calm = torch.where(keep[:, None], x, x.clamp(-1, 1))
        assert torch.equal(run(calm)[keep], y[keep])


def test_fp16_hidden_rows_past_the_range_captured_and_at_once():
    """Replays with other tokens, some past the range and some not, and two streams at a time."""
    x, router, cks, run = wide_layer(12, 1032, 520, 24, 4, 64, True, 3)
    wants = [run(torch.roll(x, k, 0)) for k in range(len(SIZES))]
    for k, w in enumerate(wants):
        assert torch.equal(torch.roll(w, -k, 0), wants[0])
    static = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = run(static)
        z = run(torch.zeros_like(static))
    for k, w in enumerate(wants):
        static.copy_(torch.roll(x, k, 0))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, w) and not z.any()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for k in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(run(x))
    torch.cuda.synchronize()
    assert all(torch.equal(v, wants[0]) for g in got for v in g)
    assert ops.device_error() == (0, 0)


@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("M", [1, 9, 16, 40, 128, 1100])
def test_large_activations(M, group, zeros):
    """Rows of 2^121, all of one sign, under codes of one sign: a group's sum passes fp32's range, the output, under scales of
    2^-20, does not."""
    K, N = 392, 200
    g = torch.Generator(device=DEV).manual_seed(M)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8) | 0xCC
    scales = ((torch.rand(N, -(-K // group), generator=g, device=DEV) + 0.5) * 2.0 ** -20).to(BF)
    ck = (codes, scales, torch.zeros(scales.shape, dtype=torch.uint8, device=DEV) if zeros else None)
    x = torch.full((M, K), 2.0 ** 121, device=DEV, dtype=BF)
    x[:, ::3] *= 0.5
    want, err = product(x.to(F64), ck, group)
    assert (want + err).amax() < torch.finfo(BF).max
    assert (product(x.to(F64), (codes, torch.ones_like(scales), ck[2]), group)[0].amin() / (K / group)) > 2.0 ** 128 or group == 64
    check(ops.w4_linear(x, ops.w4_prepare(*ck, group=group)), want, err, BF)


@pytest.mark.parametrize("M", [1, 16, 40, 1100])
def test_smallest_activations(M):
    """Rows of bf16's smallest values under large scales."""
    K, N, group = 392, 200, 64
    g = torch.Generator(device=DEV).manual_seed(M)
    codes, scales, z = checkpoint(g, (N, K), group, True, BF, DEV)
    ck = (codes, (scales.float() * 2.0 ** 100).to(BF), z)
    x = (torch.randint(-200, 201, (M, K), generator=g, device=DEV).float() * 2.0 ** -100 * 2.0 ** -33).to(BF)
    assert (x != 0).any() and x.abs().max() < 2.0 ** -125
    want, err = product(x.to(F64), ck, group)
    check(ops.w4_linear(x, ops.w4_prepare(*ck, group=group)), want, err, BF)
