"""The FP8 quantisers' quotient, q + r (x - q s) with r = fl32(1 / s) and q = fl32(x r), is the correctly rounded
fl32(x / s) for every mantissa of a 16-bit x with every scale s = fl32(max / 448) of a 16-bit maximum, and
the scale's own quotient by 448 for every finite 16-bit value: counted through on the CPU, and by the
codes that the quantiser gives on the GPU."""

import numpy as np
import pytest
import torch


def f32(v):
    return v.astype(np.float32).astype(np.float64)


def fma(a, b, c):
    """fl32(a b + c) of fp32 values held in float64: the product is exact there; where the float64 sum lies on a
    midpoint of two fp32 values, its own rounding error decides."""
    p = a * b
    t = p + c
    z = t - c
    err = (p - z) + (c - (t - z))
    mid = (t.view(np.int64) & 0x1FFFFFFF) == 0x10000000
    toward = np.where(err > 0, np.inf, -np.inf)
    return f32(np.where(mid & (err != 0), np.nextafter(t, toward), t))


def corrected(x, s, r):
    q = f32(x * r)
    return fma(fma(-q, s, x), r, q), q


@pytest.mark.parametrize("bits", [7, 10])
def test_every_pair_of_mantissas(bits):
    m = 1.0 + np.arange(2 ** bits) / 2 ** bits
    s = f32(m / 448.0)[:, None]
    got, q = corrected(np.broadcast_to(m, (m.size, m.size)).copy(), s, f32(1.0 / s))
    want = f32(m[None, :] / s)  # 24-bit operands: rounding to 53 and then 24 bits is rounding once
    assert np.array_equal(got, want)
    # the uncorrected product is more than one unit of the last place off for some pairs
    exact = m[None, :] / s
    assert (np.abs(q - exact) > np.spacing(exact.astype(np.float32)).astype(np.float64)).any()


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
def test_every_scale(kind):
    v = torch.arange(0, 0x7F80 if kind == torch.bfloat16 else 0x7C00, dtype=torch.int16).view(kind)
    a = v.double().numpy()
    got, _ = corrected(a, np.float64(448.0), np.float64(np.float32(1.0 / 448.0)))
    assert np.array_equal(got, f32(a / 448.0))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("down", [0, 1, 3, 6, 9])
def test_every_pair_through_the_quantiser(kind, down):
    """Row i holds, in every block of 128, the maximum with mantissa i and then mantissas in turn, 2^(1 + down) smaller."""
    from nvfp4_block_scaled_quant_gb300 import ops
    n = 128 if kind == torch.bfloat16 else 1024
    m = 1.0 + torch.arange(n, dtype=torch.float64, device="cuda") / n
    blocks = -(-n // 127)
    x = torch.ones(n, blocks, 128, dtype=torch.float64, device="cuda")
    x[:, :, 1:] = torch.cat([m, m])[:blocks * 127].view(blocks, 127) * 2.0 ** -down
    x[:, :, 0] = 2.0 * m[:, None]  # above every other value of the block
    x = x.view(n, blocks * 128)
    assert torch.equal(x.to(kind).double(), x)
    q, s = ops.fp8_quantize_act(x.to(kind))
    want_s = (x.view(n, blocks, 128).abs().amax(2) / 448.0).float()
    v = (x.view(n, blocks, 128) / want_s.double()[:, :, None]).float()
    assert torch.equal(s.T, want_s)
    assert torch.equal(q.view(torch.uint8), v.clamp(-448, 448).to(torch.float8_e4m3fn).view(n, -1).view(torch.uint8))
