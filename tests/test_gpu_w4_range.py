"""The operators on 4-bit weights with scales and activations at the ends of their range, against the definition in 64 bits."""

import pytest
import torch

from nvfp4_block_scaled_quant_gb300 import ops
from w4_reference import F64, check, checkpoint, moe, product

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
