"""Calls of the dense operators that are refused on a machine with a GPU (nothing is launched, and what the
call would have written is as it was), and calls with no rows, which are not."""

import pytest
import torch

from nvfp4_block_scaled_quant_gb300 import _lib, ops

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = _lib.DT_BF16


def test_quantising_into_the_activations():
    buf = torch.arange(1 << 14, device=DEV).to(torch.bfloat16)
    keep, p = buf.clone(), buf.data_ptr()
    free = torch.zeros(1 << 14, dtype=torch.uint8, device=DEV).data_ptr()
    for q, xs in ((p, free), (p + 4 * 256 * 2 - 16, free), (free, p + 1024), (free, free + 4 * 256 - 16)):
        with pytest.raises(RuntimeError, match="overlap"):
            _lib.call("nvfp4_fp8_quantize_act", p, BF, 4, 256, 256, q, xs, 4, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(buf, keep)


def test_outputs_and_workspaces_inside_inputs():
    bf = dict(dtype=torch.bfloat16, device=DEV)
    x, r = torch.ones(64, 256, **bf), torch.ones(64, 256, **bf)
    w, ws = ops.fp8_quantize_weight(torch.ones(256, 256, **bf))
    wg, wu = torch.ones(64, 256, **bf), torch.ones(256, 256, **bf)
    gate, gb = torch.ones(64, 256, **bf), torch.ones(256, **bf)
    h, gu = ops.gated_linear(x, wg, wg, save=True)
    grad_ws = gu.view(torch.uint8).view(-1)
    keep = [t.clone() for t in (x, r, wg, wu, gate, gu)]
    for call in [lambda: ops.fp8_linear(x, w, ws, out=wu[:64].view(64, 256), workspace=wu.view(torch.uint8).view(-1)),
                 lambda: ops.gated_linear(x, wu, wu, out=wu[:64]),
                 lambda: ops.gated_linear_backward(h, x, wg, wg, gu, workspace=grad_ws),
                 lambda: ops.residual_norm(x, r, gate=gate, out=gate),
                 lambda: ops.residual_norm(x, r, gamma_before=x[3], out=x)]:
        with pytest.raises(RuntimeError, match="overlap"):
            call()
    torch.cuda.synchronize()
    for a, b in zip((x, r, wg, wu, gate, gu), keep):
        assert torch.equal(a, b)


def test_inputs_that_require_grad():
    """A call that records no graph would lose their gradients without a word; under no_grad it is made, and inside an
    autograd function its forward and backward calls are."""
    bf = dict(dtype=torch.bfloat16, device=DEV)
    x, dh, w, g = torch.randn(6, 64, **bf), torch.randn(6, 16, **bf), torch.randn(16, 64, **bf), torch.randn(64, **bf)
    h, gu = ops.gated_linear(x, w, w, save=True)
    r_out, y, stats = ops.residual_norm(x, x, g, gate=g, gamma_before=g, save=True)
    xp, wp, gp, dp = (torch.nn.Parameter(t) for t in (x, w, g, dh))
    calls = [lambda: ops.gated_linear(xp, w, w), lambda: ops.gated_linear(x, wp, w), lambda: ops.gated_linear(x, w, wp),
             lambda: ops.gated_linear_backward(dp, x, w, w, gu), lambda: ops.gated_linear_backward(dh, x, wp, w, gu),
             lambda: ops.residual_norm(xp, x), lambda: ops.residual_norm(x, xp), lambda: ops.residual_norm(x, x, gp),
             lambda: ops.residual_norm(x, x, gate=gp), lambda: ops.residual_norm(x, x, gamma_before=gp),
             lambda: ops.residual_norm(xp, x, stream=torch.cuda.current_stream()),
             lambda: ops.residual_norm_backward(xp, None, x, x, stats, g, gate=g, gamma_before=g),
             lambda: ops.residual_norm_backward(x, x, x, x, stats, gp, gate=g, gamma_before=g)]
    for call in calls:
        with pytest.raises(ValueError, match="grad"):
            call()
        with torch.no_grad():
            call()

    class Gated(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, wg, wu):
            h, gu = ops.gated_linear(x, wg, wu, save=True)
            ctx.save_for_backward(x, wg, wu, gu)
            return h

        @staticmethod
        def backward(ctx, dh):
            x, wg, wu, gu = ctx.saved_tensors
            return ops.gated_linear_backward(dh, x, wg, wu, gu)

    out = Gated.apply(xp, wp, wp)
    out.backward(dh)
    dx, dwg, dwu = ops.gated_linear_backward(dh, x, w, w, gu)
    assert torch.equal(out, h) and torch.equal(xp.grad, dx) and torch.equal(wp.grad, dwg + dwu)


@pytest.mark.parametrize("K", [64, 256, 400])
def test_no_rows_through_every_call(K):
    bf = dict(dtype=torch.bfloat16, device=DEV)
    x, none = torch.empty(0, K, **bf), torch.empty(0, 1, **bf)
    w, ws = ops.fp8_quantize_weight(torch.ones(24, K, **bf))
    q, s = ops.fp8_quantize_act(x)
    assert q.shape == (0, K) and s.shape == ((K + 127) // 128, 0)
    assert ops.fp8_gemm(q, s, w, ws).shape == (0, 24) and ops.fp8_linear(x, w, ws).shape == (0, 24)
    wg = torch.ones(24, K, **bf)
    h, gu = ops.gated_linear(x, wg, wg, save=True)
    dx, dwg, dwu = ops.gated_linear_backward(h, x, wg, wg, gu)
    assert dx.shape == (0, K) and not dwg.any() and not dwu.any()
    g = torch.ones(K, **bf)
    for gate in (None, g, torch.ones(3, K, **bf), none):
        r_out, y, st = ops.residual_norm(x, x, g, gate=gate, gamma_before=g, save=True)
        df, dr, dga, dgate, dgb = ops.residual_norm_backward(r_out, y, x, x, st, g, gate=gate, gamma_before=g)
        assert r_out.shape == y.shape == df.shape == dr.shape == (0, K) and not dga.any() and not dgb.any()
        assert dgate is None if gate is None else dgate.shape == gate.shape and not dgate.any()


def test_one_row_of_scales_with_any_stride():
    """A single K block's row of scales is read as it lies, whatever its stride says."""
    bf = dict(dtype=torch.bfloat16, device=DEV)
    w, ws = ops.fp8_quantize_weight(torch.randn(24, 64, **bf))
    q, s = ops.fp8_quantize_act(torch.randn(6, 64, **bf))
    want = ops.fp8_gemm(q, s, w, ws)
    wide = torch.zeros(2, 30, device=DEV)  # rows 120 bytes apart, the first one 16-byte aligned
    wide[0, :6] = s[0]
    assert torch.equal(ops.fp8_gemm(q, wide[:1, :6], w, ws), want)


def test_gates_of_other_ranks():
    f = torch.zeros(6, 64, dtype=torch.bfloat16, device=DEV)
    for shape in ((), (1, 6, 64)):
        with pytest.raises(ValueError, match="gate"):
            ops.residual_norm(f, f, gate=torch.zeros(shape, dtype=torch.bfloat16, device=DEV))
