"""One workspace of the caller's for calls of the 4-bit linear with any number of rows."""

import pytest
import torch

from nvfp4_block_scaled_quant_gb300 import ops
from w4_reference import F64, check, checkpoint, product

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,K,group", [(1137, 2000, 32), (64, 256, 32), (4096, 1024, 128)])
def test_one_workspace(N, K, group):
    g = torch.Generator(device="cuda").manual_seed(N)
    ck = checkpoint(g, (N, K), group, True, torch.bfloat16, "cuda")
    w = ops.w4_prepare(*ck, group=group)
    x = torch.randn(2500, K, generator=g, device="cuda").bfloat16()
    ws = ops.w4_linear_workspace(2500, w)
    assert ws.numel() >= 2 * N * K
    for M in (1, 16, 40, 100, 300, 1100, 1500, 2000, 2500):
        ws.fill_(0xFF)  # it needs no initialisation
        y = ops.w4_linear(x[:M], w, workspace=ws)
        assert torch.equal(y, ops.w4_linear(x[:M], w))
        want, err = product(x[:M].to(F64), ck, group)
        check(y, want, err, x.dtype, f"{M}")


def test_small_and_foreign_workspaces():
    g = torch.Generator(device="cuda").manual_seed(1)
    w = ops.w4_prepare(*checkpoint(g, (512, 512), 64, False, torch.float16, "cuda"), group=64)
    x = torch.randn(4000, 512, generator=g, device="cuda").half()
    ws = ops.w4_linear_workspace(4000, w)
    assert ops.w4_linear_workspace(16, w).numel() == 0
    assert torch.equal(ops.w4_linear(x[:16], w, workspace=ops.w4_linear_workspace(16, w)), ops.w4_linear(x[:16], w))
    with pytest.raises(RuntimeError, match="workspace"):
        ops.w4_linear(x, w, workspace=ws[:-256])
    with pytest.raises(ValueError, match="workspace"):
        ops.w4_linear(x, w, workspace=ws.view(torch.int16))


def test_a_workspace_of_each_graph():
    """Graphs captured with workspaces of their own, replayed by turns."""
    g = torch.Generator(device="cuda").manual_seed(2)
    w = ops.w4_prepare(*checkpoint(g, (1160, 264), 128, True, torch.bfloat16, "cuda"), group=128)
    x = [torch.randn(1800, 264, generator=g, device="cuda").bfloat16() for _ in range(2)]
    want = [ops.w4_linear(v, w) for v in x]
    graphs, outs = [], []
    for v in x:
        ws = ops.w4_linear_workspace(1800, w)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(ops.w4_linear(v, w, workspace=ws))
        graphs.append((graph, ws))
    for _ in range(3):
        for graph, _ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
