"""The layer of experts on 4-bit weights at the sizes where a work item holds two or four panels and the rings have three stages:
many slots (an expert and up to eight of its tokens) for the GPU's CTAs."""

import pytest
import torch

from nvfp4_block_scaled_quant_gb300 import ops
from test_gpu_w4_moe import Layer
from test_gpu_w4_range import SIZES, wide_layer
from w4_reference import F64, check, moe

pytestmark = pytest.mark.gpu

# T, H, I, E, top k, shared expert, panels of an item of the up and of the down projection
SHAPES = [(64, 2920, 40, 300, 8, False, 1, 4),   # one K block per panel of y, 46 of them
          (64, 1544, 72, 300, 8, True, 1, 2),    # 25 panels of y
          (64, 72, 1304, 300, 8, True, 4, 1),    # 41 panels of h of one K block each
          (64, 520, 800, 300, 8, False, 2, 1),
          (64, 2632, 1304, 300, 8, True, 4, 4),  # several K blocks to a warp and item on both sides
          (59, 2056, 328, 290, 8, False, 2, 2),
          (16, 7168, 840, 384, 8, True, 2, 4)]   # a decode batch of a large model's layer


def panels_of_an_item(ids, T, shared, panels):
    """By the number of items for a CTA: one, from 8 on two, from 32 on four; not close to either border."""
    slots = int(sum(-(-int(n) // 8) for n in torch.bincount(ids.flatten()).tolist())) + (-(-T // 8) if shared else 0)
    rounds = slots * panels / (2 * torch.cuda.get_device_properties(0).multi_processor_count)
    assert all(abs(rounds / edge - 1) > 0.02 for edge in (8, 32)), rounds
    return 1 if rounds < 8 else 2 if rounds < 32 else 4


@pytest.mark.parametrize("kind,group,zeros", [("bf16", 128, False), ("fp16", 64, True), ("bf16", 32, True), ("fp16", 128, True), ("bf16", 64, False),
                                              ("fp16", 32, False)])
@pytest.mark.parametrize("T,H,I,E,topk,shared,up,down", SHAPES)
def test_items_of_several_panels(T, H, I, E, topk, shared, up, down, kind, group, zeros):
    layer = Layer(T, H, I, E, topk, shared, group, zeros, kind, seed=11)
    y = layer.run()
    ids = layer.verify(y)
    assert panels_of_an_item(ids, T, shared, -(-I // 32)) == up
    assert panels_of_an_item(ids, T, shared, -(-H // 64)) == down
    for _ in range(3):
        assert torch.equal(layer.run(), y)
    assert ops.device_error() == (0, 0)


@pytest.mark.parametrize("T,H,I,E,up,down", [(64, 72, 1304, 300, 4, 1), (64, 2920, 264, 300, 1, 4), (64, 1304, 1304, 300, 4, 2)])
def test_items_of_several_panels_past_the_range(T, H, I, E, up, down):
    """The same where panels of fp16 hidden rows pass 65504."""
    x, router, cks, run = wide_layer(T, H, I, E, 8, 64, True, 12)
    want, err, ids, _ = moe(x.to(F64), router, cks[0], cks[1], 8, 64, "silu", x.dtype, (cks[2], cks[3]))
    assert panels_of_an_item(ids, T, True, -(-I // 32)) == up
    assert panels_of_an_item(ids, T, True, -(-H // 64)) == down
    fits = want.abs() + err < 65504
    assert fits.float().mean() > 1 - 2 / len(SIZES)
    y = run(x)
    check(torch.where(fits, y, 0), torch.where(fits, want, 0), err, x.dtype)
    assert torch.equal(run(x), y)
