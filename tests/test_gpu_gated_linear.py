"""Gated linear and its gradients on the GPU against their formulas in 64 bits.

Exact cases: with gate pre-activations of 32 or more, SiLU(g) = g and SiLU'(g) = 1 exactly in fp32,
so integer inputs give integer outputs that are exact before the one rounding of the output type;
any index or layout mistake shows.  Random cases are held to bounds that count every rounding:
half a step u of the 16-bit type for the output (and, in the backward, for dg and du), and one fp32
step of the sum of absolute products for each addition of a sum.
"""

import math

import pytest
import torch

from nvfp4_block_scaled_quant_gb300 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.bfloat16, torch.float16]


def act64(g, kind):
    if kind == "silu":
        p = torch.sigmoid(g)
        return g * p, p + g * p * torch.sigmoid(-g)
    if kind == "gelu":
        p = 0.5 * torch.erfc(-g / math.sqrt(2.0))
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    b = math.sqrt(2 / math.pi)
    p = torch.sigmoid(2 * b * (g + 0.044715 * g ** 3))
    return g * p, p + g * 2 * p * (1 - p) * b * (1 + 3 * 0.044715 * g * g)


def ints(gen, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=gen, device=DEV).double()


SHAPES = [(1, 64, 8), (1, 8, 128), (3, 136, 136), (16, 512, 264), (17, 200, 72), (33, 1544, 128), (64, 256, 1000), (65, 128, 256),
          (128, 320, 384), (129, 72, 40), (200, 264, 520), (256, 512, 128), (300, 1000, 136), (513, 128, 1032), (1100, 200, 264)]


@pytest.mark.parametrize("T,H,I", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_forward_exact_integers(T, H, I, dtype):
    gen = torch.Generator(device=DEV).manual_seed(T + H + I)
    x, wg, wu = ints(gen, 0, 2, T, H), ints(gen, 0, 2, I, H), ints(gen, -1, 1, I, H)
    x[:, 0], wg[:, 0] = 8, 8  # every g is at least 64
    g, u = x @ wg.T, x @ wu.T
    h, gu = ops.gated_linear(x.to(dtype), wg.to(dtype), wu.to(dtype), save=True)
    assert torch.equal(gu[:, :I].double(), g) and torch.equal(gu[:, I:].double(), u)
    assert (g * u).abs().max() < 2 ** 24
    assert torch.equal(h, (g * u).to(dtype))
    assert torch.equal(h, ops.gated_linear(x.to(dtype), wg.to(dtype), wu.to(dtype)))
    assert ops.device_error() == (0, 0)


@pytest.mark.parametrize("T,H,I", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_backward_exact_integers(T, H, I, dtype):
    gen = torch.Generator(device=DEV).manual_seed(T * 3 + H + I)
    x, wg, wu = ints(gen, -1, 1, T, H), ints(gen, -1, 1, I, H), ints(gen, -1, 1, I, H)
    dh, u = ints(gen, -1, 1, T, I), ints(gen, -2, 2, T, I)
    g = 32 + 32 * ints(gen, 0, 1, T, I)
    dx, dwg, dwu = ops.gated_linear_backward(dh.to(dtype), x.to(dtype), wg.to(dtype), wu.to(dtype), torch.cat([g, u], 1).float())
    dg, du = dh * u, dh * g
    for got, want in ((dx, dg @ wg + du @ wu), (dwg, dg.T @ x), (dwu, du.T @ x)):
        assert torch.equal(got, want.to(dtype))
    assert ops.device_error() == (0, 0)


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,I", [(1, 1536, 264), (20, 512, 136), (333, 264, 200), (520, 512, 1000)])
def test_random_forward_and_gradients(T, H, I, dtype, kind):
    gen = torch.Generator(device=DEV).manual_seed(T + I)
    x = torch.randn(T, H, generator=gen, device=DEV).to(dtype)
    wg, wu = ((torch.randn(I, H, generator=gen, device=DEV) * 2 * H ** -0.5).to(dtype) for _ in range(2))
    dh = torch.randn(T, I, generator=gen, device=DEV).to(dtype)
    h, gu = ops.gated_linear(x, wg, wu, activation=kind, save=True)
    dx, dwg, dwu = ops.gated_linear_backward(dh, x, wg, wu, gu, activation=kind)

    X, G, U, D = x.double(), wg.double(), wu.double(), dh.double()
    g, u = X @ G.T, X @ U.T
    a, da = act64(g, kind)
    e, o = 2.0 ** -23, torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * o
    eg, eu = H * e * (X.abs() @ G.abs().T), H * e * (X.abs() @ U.abs().T)
    assert ((gu[:, :I] - g).abs() <= eg).all() and ((gu[:, I:] - u).abs() <= eu).all()
    # |act'| <= 1.2, |act''| <= 1.2; 16 fp32 steps for the activation itself (its p is at most 1)
    ea, eda = 1.2 * eg + 16 * e * (g.abs() + 1), 1.2 * eg + 16 * e * (g.abs() + 1) * 1.3
    eh = ea * (u.abs() + eu) + a.abs() * eu
    assert ((h - a * u).abs() <= (1 + o) * eh + o * (a * u).abs() + tiny).all()
    dg, du = D * u * da, D * a
    edg = D.abs() * (eda * (u.abs() + eu) + da.abs() * eu + 4 * e * (u * da).abs())
    edu = D.abs() * (ea + 4 * e * a.abs())
    edg, edu = (1 + o) * edg + o * dg.abs() + tiny, (1 + o) * edu + o * du.abs() + tiny

    def held(got, want, err, mag, n):
        err = err + n * e * mag
        off = (got.double() - want).abs()
        assert (off <= (1 + o) * err + o * want.abs() + tiny).all()
        # roundings of half a step at most, in dg or du and in the output: in the 2-norm, where they
        # do not line up, under two of them
        assert off.norm() <= 2 * o * want.norm()

    held(dx, dg @ G + du @ U, edg @ G.abs() + edu @ U.abs(), dg.abs() @ G.abs() + du.abs() @ U.abs(), 2 * I)
    held(dwg, dg.T @ X, edg.T @ X.abs(), dg.abs().T @ X.abs(), T)
    held(dwu, du.T @ X, edu.T @ X.abs(), du.abs().T @ X.abs(), T)


def test_gradient_against_differences():
    """The 64-bit formulas the other tests use are the derivative: central differences of the loss
    sum(h dh), whose error is O(d^2) = 1e-8 of the third derivative plus 1e-16 / d of rounding."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    T, H, I = 5, 16, 8
    x, wg, wu, dh = (torch.randn(*s, generator=gen, device=DEV).bfloat16() for s in ((T, H), (I, H), (I, H), (T, I)))
    for kind in ("silu", "gelu", "gelu_tanh"):
        _, gu = ops.gated_linear(x, wg, wu, activation=kind, save=True)
        grads = ops.gated_linear_backward(dh, x, wg, wu, gu, activation=kind)
        base = [t.double() for t in (x, wg, wu)]

        def loss(p):
            return (act64(p[0] @ p[1].T, kind)[0] * (p[0] @ p[2].T) * dh.double()).sum()

        for k in range(3):
            v = torch.randn(base[k].shape, generator=gen, device=DEV, dtype=torch.float64)
            d = 1e-4
            up, down = ([b + s * d * v if i == k else b for i, b in enumerate(base)] for s in (1, -1))
            diff = (loss(up) - loss(down)) / (2 * d)
            # every element of the gradient is within four half steps (two roundings; sums of a few terms)
            tol = 4 * 2.0 ** -8 * (grads[k].double() * v).abs().sum() + 1e-4 * diff.abs() + 1e-3
            assert (diff - (grads[k].double() * v).sum()).abs() <= tol


@pytest.mark.parametrize("T", [4, 300])
def test_strides_and_partial_gradients(T):
    gen = torch.Generator(device=DEV).manual_seed(T)
    bx, bd = torch.randn(T, 300, generator=gen, device=DEV).bfloat16(), torch.randn(T, 160, generator=gen, device=DEV).bfloat16()
    bx, bd = torch.cat([bx, bx[:, :4]], 1), bd
    x, dh = bx[:, 8:8 + 136], bd[:, 16:16 + 72]
    wg, wu = (torch.randn(72, 136, generator=gen, device=DEV).bfloat16() for _ in range(2))
    h, gu = ops.gated_linear(x, wg, wu, save=True)
    h2, gu2 = ops.gated_linear(x.contiguous(), wg, wu, save=True)
    assert torch.equal(h, h2) and torch.equal(gu, gu2)
    full = ops.gated_linear_backward(dh.contiguous(), x.contiguous(), wg, wu, gu)
    for got, want in zip(ops.gated_linear_backward(dh, x, wg, wu, gu), full):
        assert torch.equal(got, want)
    a = ops.gated_linear_backward(dh, x, wg, wu, gu, need_dw=False)
    b = ops.gated_linear_backward(dh, x, wg, wu, gu, need_dx=False)
    assert torch.equal(a[0], full[0]) and a[1] is None and b[0] is None and torch.equal(b[1], full[1]) and torch.equal(b[2], full[2])
    out = torch.full((T + 1, 72), 5.0, dtype=torch.bfloat16, device=DEV)
    ops.gated_linear(x, wg, wu, out=out[:T])
    assert torch.equal(out[:T], h) and (out[T] == 5.0).all()


def test_no_rows():
    x, w = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), torch.ones(8, 64, dtype=torch.bfloat16, device=DEV)
    h, gu = ops.gated_linear(x, w, w, save=True)
    assert h.shape == (0, 8) and gu.shape == (0, 16)
    dx, dwg, dwu = ops.gated_linear_backward(h, x, w, w, gu)
    assert dx.shape == (0, 64) and (dwg == 0).all() and (dwu == 0).all()


@pytest.mark.parametrize("T", [2, 300])
def test_capture_of_forward_and_backward(T):
    gen = torch.Generator(device=DEV).manual_seed(T)
    x, dh = (torch.randn(T, n, generator=gen, device=DEV).bfloat16() for n in (256, 128))
    wg, wu = (torch.randn(128, 256, generator=gen, device=DEV).bfloat16() for _ in range(2))

    def step(x):
        h, gu = ops.gated_linear(x, wg, wu, save=True)
        return (h, *ops.gated_linear_backward(dh, x, wg, wu, gu))

    step(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x)
    x2 = torch.randn(T, 256, generator=gen, device=DEV).bfloat16()
    want = step(x2)
    x.copy_(x2)
    graph.replay()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_refusals():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(16, 64, dtype=torch.bfloat16, device=DEV)
    h, gu = ops.gated_linear(x, w, w, save=True)
    for f in [lambda: ops.gated_linear(x, w, w[:8]), lambda: ops.gated_linear(x, w.half(), w.half()),
              lambda: ops.gated_linear(x.float(), w.float(), w.float()), lambda: ops.gated_linear(x, w, w, activation="relu"),
              lambda: ops.gated_linear(x, w.T, w.T), lambda: ops.gated_linear_backward(h[:2], x, w, w, gu),
              lambda: ops.gated_linear_backward(h, x, w, w, gu.bfloat16()), lambda: ops.gated_linear(x.cpu(), w, w),
              lambda: ops.gated_linear_backward(h.half(), x, w, w, gu)]:
        with pytest.raises(ValueError):
            f()
    for f in [lambda: ops.gated_linear(x[:, :60], w[:, :60].contiguous(), w[:, :60].contiguous()),
              lambda: ops.gated_linear(x, w[:12], w[:12]),
              lambda: ops.gated_linear_backward(h, x, w, w, gu, workspace=torch.empty(128, dtype=torch.uint8, device=DEV))]:
        with pytest.raises(RuntimeError, match="nvfp4 status"):
            f()
