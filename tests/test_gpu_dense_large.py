"""The dense operators on tensors of more than 2^31 elements: the last rows, whose offsets pass 32 bits,
against a call on those rows alone.  A row's result does not depend on the other rows, and the sums of
these shapes run in the same order in both calls, so the bits agree."""

import pytest
import torch

from nvfp4_block_scaled_quant_gb300 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"
M, K, TAIL = 300_000, 8192, 4096  # 2.46e9 elements


@pytest.fixture(autouse=True)
def room():
    free, _ = torch.cuda.mem_get_info()
    if free < 100 << 30:
        pytest.skip("needs 100 GB of device memory")
    yield
    torch.cuda.empty_cache()


def rows(seed, m=M, k=K):
    """(m, k) bf16 values, made in place (no 32-bit copy of the whole tensor)."""
    return torch.empty(m, k, dtype=torch.bfloat16, device=DEV).normal_(generator=torch.Generator(device=DEV).manual_seed(seed))


def test_residual_norm_and_gradients():
    f, r, dy = rows(1), rows(2), rows(3)
    ga, gb = (1 + 0.1 * torch.randn(2, K, device=DEV)).bfloat16()
    out, y, st = ops.residual_norm(f, r, ga, gamma_before=gb, save=True)
    df, dr, *_ = ops.residual_norm_backward(dy, dy, f, r, st, ga, gamma_before=gb)
    tail = [t[-TAIL:] for t in (f, r, dy)]
    out2, y2, st2 = ops.residual_norm(tail[0], tail[1], ga, gamma_before=gb, save=True)
    df2, dr2, *_ = ops.residual_norm_backward(tail[2], tail[2], tail[0], tail[1], st2, ga, gamma_before=gb)
    for big, small in ((out, out2), (y, y2), (st, st2), (df, df2), (dr, dr2)):
        assert torch.equal(big[-TAIL:], small)
    assert ops.device_error() == (0, 0)


def test_fp8_linear():
    x = rows(4)
    q, s = ops.fp8_quantize_act(x)
    q2, s2 = ops.fp8_quantize_act(x[-TAIL:])
    assert torch.equal(q[-TAIL:].view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s[:, -TAIL:], s2)
    del x, q, s
    w, ws = ops.fp8_quantize_weight(rows(5, K, 128))
    x = rows(6, M, 128)
    y = ops.fp8_linear(x, w, ws)
    assert torch.equal(y[-TAIL:], ops.fp8_linear(x[-TAIL:], w, ws))
    assert ops.device_error() == (0, 0)


def test_gated_linear_and_gradients():
    H = 64
    x, wg, wu, dh = rows(7, M, H), rows(8, K, H), rows(9, K, H), rows(10)
    h, gu = ops.gated_linear(x, wg, wu, save=True)
    dx, dwg, dwu = ops.gated_linear_backward(dh, x, wg, wu, gu)
    xt, dht = x[-TAIL:], dh[-TAIL:]
    h2, gu2 = ops.gated_linear(xt, wg, wu, save=True)
    dx2, _, _ = ops.gated_linear_backward(dht, xt, wg, wu, gu2, need_dw=False)
    for big, small in ((h, h2), (gu, gu2), (dx, dx2)):
        assert torch.equal(big[-TAIL:], small)
    # four rows of the weight gradients over all tokens, in 64 bits; two roundings of half a step that do not
    # line up (dg or du and the output), as in the small cases
    c = slice(K - 4, K)
    g, u, d = gu[:, :K][:, c].double(), gu[:, K:][:, c].double(), dh[:, c].double()
    p = torch.sigmoid(g)
    for got, dz in ((dwg, d * u * (p + g * p * (1 - p))), (dwu, d * g * p)):
        want = dz.T @ x.double()
        assert (got[c].double() - want).norm() <= 2 * 2.0 ** -8 * want.norm()
    assert ops.device_error() == (0, 0)
