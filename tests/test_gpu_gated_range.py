"""Gated linear's gradients where dg = dh u act'(g) and du = dh act(g) leave fp16's range or its normal numbers
though the gradients do not, and NaN and infinities, against the formulas in 64 bits.

Every element of dg and du is off by a few fp32 steps, half a step o = eps / 2 of the type and 2^-39 of the
largest one of both (the end of fp16 below the power of two that they are stored with); a sum of n
products adds n fp32 steps of the sum of their absolute values, an output half a step of its own (o of the
value, or half of the smallest step)."""

import pytest
import torch

from nvfp4_block_scaled_quant_gb300 import ops
from tests.test_gpu_gated_linear import act64

pytestmark = pytest.mark.gpu
DEV = "cuda"
KINDS = ["silu", "gelu", "gelu_tanh"]


def gradients(T, H, I, dtype, kind, dh_size, u_size, w_size, x_size, seed, rows=None):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=gen, device=DEV)

    x, wg, wu = (x_size * normal(T, H)).to(dtype), (w_size * normal(I, H)).to(dtype), (w_size * normal(I, H)).to(dtype)
    dh = dh_size * normal(T, I)
    if rows is not None:  # sizes by token
        dh = dh * rows[:, None]
    dh = dh.to(dtype)
    gu = torch.cat([3 * normal(T, I), u_size * normal(T, I)], 1)
    got = ops.gated_linear_backward(dh, x, wg, wu, gu, activation=kind)

    X, G, U, D, g, u = x.double(), wg.double(), wu.double(), dh.double(), gu[:, :I].double(), gu[:, I:].double()
    a, da = act64(g, kind)
    e, o = 2.0 ** -23, torch.finfo(dtype).eps / 2
    dg, du = D * u * da, D * a
    floor = 2.0 ** -39 * torch.maximum(dg.abs().max(), du.abs().max())
    # |act'| <= 1.2; 16 fp32 steps for the activation and its derivative, four for the products
    edg = D.abs() * u.abs() * (16 * e * (g.abs() + 1) * 1.3 + 4 * e * da.abs())
    edu = D.abs() * (16 * e * (g.abs() + 1) + 4 * e * a.abs())
    edg, edu = (1 + o) * edg + o * dg.abs() + floor, (1 + o) * edu + o * du.abs() + floor
    want = (dg @ G + du @ U, dg.T @ X, du.T @ X)
    errs = (edg @ G.abs() + edu @ U.abs() + 2 * I * e * (dg.abs() @ G.abs() + du.abs() @ U.abs()),
            edg.T @ X.abs() + T * e * (dg.abs().T @ X.abs()), edu.T @ X.abs() + T * e * (du.abs().T @ X.abs()))
    return got, want, errs


def held(got, want, errs):
    half = torch.finfo(got[0].dtype).smallest_normal * torch.finfo(got[0].dtype).eps / 2  # of the smallest step
    for y, w, err in zip(got, want, errs):
        o = torch.finfo(y.dtype).eps / 2
        assert (w.abs() < torch.finfo(y.dtype).max).all()  # the case: finite gradients
        off = (y.double() - w).abs()
        assert (off <= (1 + o) * err + o * w.abs() + half).all()
        # two roundings that do not line up, in the 2-norm
        assert off.norm() <= 2 * o * w.norm() + half * w.numel() ** 0.5


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,H,I", [(1, 64, 8), (40, 136, 264), (333, 264, 200), (700, 512, 520)])
@pytest.mark.parametrize("dh_size,u_size,w_size,x_size", [
    (2000.0, 50.0, 0.005, 0.005),   # a scaled loss: |dg| up to 4e5
    (10000.0, 300.0, 1e-4, 1e-4),   # |dg| up to 1e7
    (1e-4, 1.0, 1.0, 1.0),
    (1e-5, 1.0, 1.0, 1.0),          # ordinary gradients without scaling: dg below the normal numbers
    (2e-6, 0.05, 30.0, 30.0)])
def test_gradients_near_the_ends_of_fp16(T, H, I, dtype, kind, dh_size, u_size, w_size, x_size):
    held(*gradients(T, H, I, dtype, kind, dh_size, u_size, w_size, x_size, seed=T + I))
    assert ops.device_error() == (0, 0)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_tokens_of_very_different_size(dtype):
    rows = torch.logspace(4, -4, 90, device=DEV)  # |dh| from 1e4 to 1e-4
    held(*gradients(90, 264, 200, dtype, "silu", 1.0, 1.0, 0.02, 0.02, seed=7, rows=rows))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_no_gradient_at_all(dtype):
    got, _, _ = gradients(30, 64, 16, dtype, "silu", 0.0, 1.0, 1.0, 1.0, seed=1)
    assert all((t == 0).all() for t in got)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("T", [9, 300])
def test_a_non_finite_gradient_stays_in_its_row_and_channel(dtype, bad, T):
    gen = torch.Generator(device=DEV).manual_seed(T)
    x, dh = (torch.randn(T, n, generator=gen, device=DEV).to(dtype) for n in (72, 40))
    wg, wu = (torch.randn(40, 72, generator=gen, device=DEV).to(dtype) for _ in range(2))
    _, gu = ops.gated_linear(x, wg, wu, save=True)
    clean = ops.gated_linear_backward(dh, x, wg, wu, gu)
    dh[4, 3] = bad
    dx, dwg, dwu = ops.gated_linear_backward(dh, x, wg, wu, gu)
    tokens, channels = [t for t in range(T) if t != 4], [i for i in range(40) if i != 3]
    assert not torch.isfinite(dx[4]).any() and not torch.isfinite(dwg[3]).any() and not torch.isfinite(dwu[3]).any()
    assert torch.equal(dx[tokens], clean[0][tokens])
    assert torch.equal(dwg[channels], clean[1][channels]) and torch.equal(dwu[channels], clean[2][channels])


@pytest.mark.parametrize("T", [5, 40, 300])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_non_finite_token_stays_in_its_row(T, bad):
    gen = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn(T, 136, generator=gen, device=DEV).bfloat16()
    wg, wu = (torch.randn(264, 136, generator=gen, device=DEV).bfloat16() for _ in range(2))
    clean = ops.gated_linear(x, wg, wu)
    x[2, 7] = bad
    h = ops.gated_linear(x, wg, wu)
    rest = [t for t in range(T) if t != 2]
    assert torch.equal(h[rest], clean[rest])
    # NaN everywhere, or the infinities (and 0 inf = NaN) of the activation at +-inf
    if bad != bad:
        assert torch.isnan(h[2]).all()
    else:
        assert not torch.isfinite(h[2]).any()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [50.0, 1e4, 1e10, 1.5e19, 3e19, 1e30])
def test_huge_pre_activations(kind, size):
    """act'(g) is 1 or 0 there: no product inside it may leave fp32's range."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    T, H, I = 20, 64, 16
    x, wg, wu, dh, u = (torch.randn(*s, generator=gen, device=DEV).bfloat16() for s in ((T, H), (I, H), (I, H), (T, I), (T, I)))
    g = size * (torch.randint(0, 2, (T, I), generator=gen, device=DEV) * 2.0 - 1)
    got = ops.gated_linear_backward(dh, x, wg, wu, torch.cat([g, u.float()], 1), activation=kind)
    a, da = act64(g.double(), kind)
    X, G, U, D = x.double(), wg.double(), wu.double(), dh.double()
    dg, du = D * u.double() * da, D * a
    want = (dg @ G + du @ U, dg.T @ X, du.T @ X)
    mags = (dg.abs() @ G.abs() + du.abs() @ U.abs(), dg.abs().T @ X.abs(), du.abs().T @ X.abs())
    o, e = 2.0 ** -8, 2.0 ** -23
    for y, w, mag in zip(got, want, mags):
        assert torch.isfinite(y).all()
        # half a step of dg or du and of the output; 16 fp32 steps of an activation, 2 I or T of a sum
        assert ((y.double() - w).abs() <= (1 + o) * (o + (16 + 2 * I + T) * e) * mag + o * w.abs()).all()


@pytest.mark.parametrize("T", [6, 300])
def test_captured_gradients_follow_the_size_of_the_data(T):
    """The power of two is chosen on the device: a replay on much larger or smaller gradients gives the bits of a
    call on them; also on another stream, with a workspace that both calls share."""
    gen = torch.Generator(device=DEV).manual_seed(T)
    x, dh = ((torch.randn(T, n, generator=gen, device=DEV) * 2.0 ** -4).half() for n in (136, 72))
    wg, wu = ((torch.randn(72, 136, generator=gen, device=DEV) * 2.0 ** -6).half() for _ in range(2))
    _, gu = ops.gated_linear(x, wg, wu, save=True)
    gu[:, 72:] += 3.0
    first = dh.clone()
    graph = torch.cuda.CUDAGraph()
    ops.gated_linear_backward(dh, x, wg, wu, gu)
    with torch.cuda.graph(graph):
        got = ops.gated_linear_backward(dh, x, wg, wu, gu)
    from nvfp4_block_scaled_quant_gb300 import _lib
    work = torch.empty(_lib.lib().nvfp4_gated_linear_backward_workspace_bytes_dt(T, 72, _lib.DT_FP16), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    for power in (0, 16, -8, 3):
        dh.copy_((first.double() * 2.0 ** power).half())
        want = ops.gated_linear_backward(dh, x, wg, wu, gu, workspace=work)
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        other = ops.gated_linear_backward(dh, x, wg, wu, gu, workspace=work, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        for a, b, c in zip(got, want, other):
            assert torch.isfinite(b).all() and b.any() and torch.equal(a, b) and torch.equal(c, b)


def test_workspace_by_type():
    from nvfp4_block_scaled_quant_gb300 import _lib
    f = _lib.lib().nvfp4_gated_linear_backward_workspace_bytes_dt
    x, w = torch.zeros(4, 64, dtype=torch.float16, device=DEV), torch.zeros(16, 64, dtype=torch.float16, device=DEV)
    h, gu = ops.gated_linear(x, w, w, save=True)
    need = f(4, 16, _lib.DT_FP16)
    assert need == f(4, 16, _lib.DT_BF16) + 4352
    ops.gated_linear_backward(h, x, w, w, gu, workspace=torch.empty(need, dtype=torch.uint8, device=DEV))
    with pytest.raises(RuntimeError, match="nvfp4 status 4"):
        ops.gated_linear_backward(h, x, w, w, gu, workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))
