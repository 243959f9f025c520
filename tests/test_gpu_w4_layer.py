"""The operators on 4-bit weights as a decode step uses them: together, captured, on several streams, beside the
framework's other operators, and their refusals on a machine with a GPU."""

import pytest
import torch

from nvfp4_block_scaled_quant_gb300 import _lib, ops
from w4_reference import F64, check, checkpoint, half_step, moe, product

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Block:
    """A layer around its attention: an 8-bit projection in, a 4-bit projection out, the experts, and the norms between
    them.  The attention itself is left out: the projection's output stands for it."""

    def __init__(self, H=512, I=160, E=24, topk=3, A=384, dt=torch.bfloat16, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.topk, self.dt = topk, dt

        def normal(*shape):
            return torch.randn(*shape, generator=g, device=DEV)

        self.g1, self.g2 = (1 + 0.1 * normal(2, H)).to(dt)
        self.q = ops.fp8_quantize_weight((normal(A, H) * H ** -0.5).to(dt))
        self.o_ck = checkpoint(g, (H, A), 64, True, dt, DEV)
        self.o = ops.w4_prepare(*self.o_ck, group=64)
        self.router = (normal(E, H) * H ** -0.5).to(dt)
        self.ck = [checkpoint(g, s, 32, False, dt, DEV) for s in ((E, 2 * I, H), (E, H, I), (2 * I, H), (H, I))]
        self.w13, self.w2, self.s13, self.s2 = (ops.w4_prepare(*c, group=32, gated=i % 2 == 0) for i, c in enumerate(self.ck))

    def __call__(self, f, r, keep=None):
        """f: the last block's output, r: the fp32 residual stream; returns the same of this layer."""
        r1, q, s, _ = ops.residual_norm_fp8(f, r, self.g1)
        a = ops.fp8_gemm(q, s, *self.q, dtype=self.dt)
        o = ops.w4_linear(a, self.o)
        r2, q2, s2, y = ops.residual_norm_fp8(o, r1, self.g2, want_y=True)
        out = ops.w4_moe(y, self.router, self.w13, self.w2, self.topk, shared13=self.s13, shared2=self.s2)
        if keep is not None:
            keep.update(q=q, s=s, a=a, o=o, r1=r1, r2=r2, y=y, q2=q2, s2=s2)
        return out, r2


def inputs(T, H=512, seed=1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(T, H, generator=g, device=DEV).bfloat16(), torch.randn(T, H, generator=g, device=DEV)


@pytest.mark.parametrize("T", [1, 5, 40, 64])
def test_each_step_of_a_layer(T):
    b, kept = Block(), {}
    f, r = inputs(T)
    out, r2 = b(f, r, kept)
    assert torch.equal(r2, kept["r2"])
    assert torch.equal(kept["r1"], (r + f.float()))
    want, err = product(kept["a"].to(F64), b.o_ck, 64)
    check(kept["o"], want, err, b.dt, "4-bit projection")
    assert torch.equal(kept["y"], ops.residual_norm(kept["o"], kept["r1"], gamma_before=b.g2)[1])
    # the same y in 8 bits: within half a step of e4m3 and y's own rounding
    sc = kept["s2"].T.repeat_interleave(128, dim=1)[:, :512].double()
    off = (kept["q2"].double() * sc - kept["y"].double()).abs()
    assert (off <= torch.maximum(2.0 ** -4 * kept["y"].double().abs(), 2.0 ** -10 * sc) * 1.01 + half_step(b.dt) * kept["y"].double().abs()).all()
    one = [tuple(None if v is None else v for v in c) for c in b.ck]
    want, err, _, sure = moe(kept["y"].to(F64), b.router, one[0], one[1], b.topk, 32, "silu", b.dt, (one[2], one[3]))
    check(out, want, err, b.dt, "experts" if sure else "experts (their choice may hang on the sums' order)")


def test_layers_in_a_graph_and_on_streams():
    """Three layers one after the other, captured and replayed on new inputs, equal to eager calls; two such chains on
    two streams at once."""
    layers = [Block(seed=s) for s in range(3)]
    ins = [inputs(7, seed=s) for s in range(4)]

    def chain(f, r):
        for b in layers:
            f, r = b(f, r)
        return f, r

    wants = [chain(*i) for i in ins]
    static = [t.clone() for t in ins[0]]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(*static)
    for _ in range(2):
        for i, want in zip(ins, wants):
            for s, t in zip(static, i):
                s.copy_(t)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(u, v) for u, v in zip(got, want))
    streams = [torch.cuda.Stream() for _ in range(2)]
    results = [[], []]
    for _ in range(5):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                results[k].append(chain(*ins[k]))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(u, v) for res in results[k] for u, v in zip(res, wants[k]))
    assert ops.device_error() == (0, 0)


@pytest.mark.parametrize("M", [1, 3, 16, 17, 100, 1500])
def test_linear_beside_other_launches(M):
    """Back to back with the kernels that start early and those on CTA pairs, on one stream and on two."""
    g = torch.Generator(device=DEV).manual_seed(M)
    K, N = 1024, 768
    ck = checkpoint(g, (N, K), 128, False, torch.bfloat16, DEV)
    w = ops.w4_prepare(*ck)
    x = torch.randn(M, K, generator=g, device=DEV).bfloat16()
    wq, ws = ops.fp8_quantize_weight(torch.randn(K, N, generator=g, device=DEV).bfloat16())
    want = ops.w4_linear(x, w)
    back = ops.fp8_linear(want, wq, ws)
    again = ops.w4_linear(back, w)
    verify, err = product(x.to(F64), ck, 128)
    check(want, verify, err, torch.bfloat16)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(10):
        y = ops.w4_linear(x, w)
        with torch.cuda.stream(side):
            z = ops.w4_linear(x, w)
        b = ops.fp8_linear(y, wq, ws)
        a = ops.w4_linear(b, w)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(z, want) and torch.equal(b, back) and torch.equal(a, again)
    assert ops.device_error() == (0, 0)


def test_the_token_counts_that_change_kernels():
    """Rows around each change of kernel and tile, alone and among others: the same values within the bounds."""
    g = torch.Generator(device=DEV).manual_seed(12)
    K, N = 640, 320
    ck = checkpoint(g, (N, K), 32, True, torch.float16, DEV)
    w = ops.w4_prepare(*ck, group=32)
    x = torch.randn(2100, K, generator=g, device=DEV).half()
    want, err = product(x.to(F64), ck, 32)
    for M in (1, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1024, 1025, 2048, 2100):
        check(ops.w4_linear(x[:M], w), want[:M], err[:M], torch.float16, f"{M} rows")


@pytest.mark.parametrize("M,K,N", [(20, 7168, 2048), (300, 2000, 1137), (900, 2048, 4096)])
def test_every_group_size_of_a_larger_product(M, K, N):
    for group in (32, 64, 128):
        g = torch.Generator(device=DEV).manual_seed(group)
        ck = checkpoint(g, (N, K), group, group != 64, torch.bfloat16, DEV)
        x = torch.randn(M, K, generator=g, device=DEV).bfloat16()
        want, err = product(x.to(F64), ck, group)
        y = ops.w4_linear(x, ops.w4_prepare(*ck, group=group))
        check(y, want, err, torch.bfloat16, f"group {group}")


def test_activations_of_any_size():
    """Rows of the smallest and largest values, one large element among small ones, rows of zeros; nothing may leak from row to row."""
    g = torch.Generator(device=DEV).manual_seed(3)
    K, N = 384, 96
    for dt, sizes in ((torch.bfloat16, (1e-38, 1e-30, 1e-10, 1.0, 1e10, 1e30)), (torch.float16, (1e-6, 1e-4, 1.0, 2e4))):
        ck = checkpoint(g, (N, K), 64, True, dt, DEV)
        w = ops.w4_prepare(*ck, group=64)
        for M in (1, 9, 40):
            x = torch.randn(M, K, generator=g, device=DEV)
            x = (x * torch.tensor(sizes, device=DEV)[torch.arange(M, device=DEV) % len(sizes)][:, None]).to(dt)
            x[M // 2] = 0
            x[M - 1, 7] = torch.finfo(dt).max / 4096
            y = ops.w4_linear(x, w)
            fine = torch.isfinite(x).all(dim=1)  # 2e4 times a normal value past 3.3 is an infinity in fp16
            assert not torch.isfinite(y[~fine]).any()
            want, err = product(x[fine].to(F64), ck, 64)
            fits = want.abs() + err < torch.finfo(dt).max
            # sums of subnormal size: fp32's own smallest step, once per step of the sum
            check(torch.where(fits, y[fine], 0), torch.where(fits, want, 0), err + 64 * 2.0 ** -149, dt, f"{dt} {M}")


def test_experts_of_any_size():
    """Tokens of very different sizes through the same experts."""
    b = Block(seed=5)
    f, _ = inputs(6, seed=6)
    x = (f.float() * torch.tensor([1e-6, 1e-3, 1.0, 30.0, 0.0, 1e3], device=DEV)[:, None]).bfloat16()
    y = ops.w4_moe(x, b.router, b.w13, b.w2, b.topk, shared13=b.s13, shared2=b.s2)
    want, err, _, _ = moe(x.to(F64), b.router, b.ck[0], b.ck[1], b.topk, 32, "silu", b.dt, (b.ck[2], b.ck[3]))
    check(y, want, err, b.dt)


def test_refusals():
    bf = dict(dtype=torch.bfloat16, device=DEV)
    codes, scales = torch.zeros(64, 64, dtype=torch.uint8, device=DEV), torch.ones(64, 1, **bf)
    w = ops.w4_prepare(codes, scales)
    gated = ops.w4_prepare(codes, scales, gated=True)
    x = torch.zeros(4, 128, **bf)
    for call, match in [(lambda: ops.w4_prepare(codes, scales, group=48), "group"), (lambda: ops.w4_prepare(codes, scales, group=32), "scales"),
                        (lambda: ops.w4_prepare(codes, scales.float()), "scales"), (lambda: ops.w4_prepare(codes[0], scales), "codes"),
                        (lambda: ops.w4_prepare(codes, scales, torch.zeros(64, 1, device=DEV)), "zeros"),
                        (lambda: ops.w4_prepare(codes.t(), scales), "contiguous|scales"),
                        (lambda: ops.w4_linear(x, gated), "expected"), (lambda: ops.w4_linear(x.half(), w), "expected"),
                        (lambda: ops.w4_linear(x[:, :64], w), "expected"), (lambda: ops.w4_linear(x.t().contiguous().t(), w), "contiguous"),
                        (lambda: ops.w4_linear(x, w, out=torch.zeros(4, 63, **bf)), "out"),
                        (lambda: ops.w4_linear(torch.nn.Parameter(x), w), "grad"),
                        (lambda: ops.w4_linear(x.cpu(), w), "devices"), (lambda: ops.w4_linear(x, w, stream=torch.cuda.Stream(), out=x.cpu()), "devices")]:
        with pytest.raises(ValueError, match=match):
            call()
    b = Block()
    f, r = inputs(4)
    for call, match in [(lambda: ops.w4_moe(f, b.router[:, :64], b.w13, b.w2, 2), "router"), (lambda: ops.w4_moe(f, b.router, b.w2, b.w13, 2), "holds"),
                        (lambda: ops.w4_moe(f, b.router, b.w13, b.w2, 2, shared13=b.s13), "together"),
                        (lambda: ops.w4_moe(f, b.router, b.w13, b.w2, 2, shared13=b.s2, shared2=b.s13), "holds"),
                        (lambda: ops.w4_moe(f, b.router, b.w13, b.w2, 2, activation="relu"), "activation"),
                        (lambda: ops.residual_norm_fp8(f, r, None), "gamma_before|grad|NULL|shape"),
                        (lambda: ops.residual_norm_fp8(torch.nn.Parameter(f), r, b.g1), "grad")]:
        with pytest.raises((ValueError, RuntimeError), match=match):
            call()
    for call, status in [(lambda: ops.w4_moe(f, b.router, b.w13, b.w2, 25), 2), (lambda: ops.w4_moe(torch.zeros(65, 512, **bf), b.router, b.w13, b.w2, 2), 2),
                         (lambda: ops.w4_moe(f, b.router, b.w13, b.w2, 2, workspace=torch.zeros(64, dtype=torch.uint8, device=DEV)), 4),
                         (lambda: ops.w4_linear(f[:, :384], b.o, out=b.o.data.view(torch.bfloat16)[:2048].view(4, 512)), 1)]:
        with pytest.raises(_lib.Nvfp4Error) as e:
            call()
        assert e.value.status == status
    torch.cuda.synchronize()
    assert ops.device_error() == (0, 0)
