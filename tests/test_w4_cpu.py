"""CPU checks of the operators on 4-bit weights and of the residual norm with an 8-bit output: the C ABI refuses bad
arguments on the host, before any device is touched, with the right status and a message; sizes of prepared weights and
workspaces; the torch layer's refusals; the arithmetic that the kernels' exactness rests on."""

import ctypes
import dataclasses

import numpy as np
import pytest
import torch

from nvfp4_block_scaled_quant_gb300 import _lib, ops
from nvfp4_block_scaled_quant_gb300 import build as B
from test_dense_cpu import changed, refuses

P = 1 << 20  # an aligned address that is never used: validation fails first
BF, HF, F32 = _lib.DT_BF16, _lib.DT_FP16, _lib.DT_FP32
NO_DEVICE = (_lib.ERR_CUDA, _lib.ERR_UNSUPPORTED_DEVICE)


@pytest.fixture(scope="module")
def L():
    B.build()
    return _lib.lib()


# ---------------------------------------------------------------- refusals of the C entry points

def test_prepare(L):
    a = dict(codes=P, scales=2 * P, zeros=3 * P, dtype=BF, G=2, N=64, K=256, group=128, gated=0, out=4 * P, stream=None)
    for kw, st in [(dict(G=0), 1), (dict(N=0), 1), (dict(K=-8), 1), (dict(dtype=F32), 1), (dict(dtype=7), 1), (dict(group=16), 1), (dict(group=0), 1),
                   (dict(codes=None), 1), (dict(scales=None), 1), (dict(out=None), 1), (dict(K=252), 2), (dict(N=65, gated=1), 2),
                   (dict(N=1 << 24), 2), (dict(K=1 << 24), 2), (dict(G=1 << 23, N=1 << 12, K=1 << 12), 2), (dict(codes=P + 2), 3),
                   (dict(scales=2 * P + 1), 3), (dict(out=4 * P + 8), 3)]:
        refuses(L, "nvfp4_w4_prepare", changed(a, **kw), st)


@pytest.mark.parametrize("G,N,K,group,zeros,gated", [(1, 1, 8, 32, 0, 0), (3, 64, 128, 64, 1, 0), (2, 65, 136, 128, 1, 0), (4, 66, 256, 32, 0, 1),
                                                     (384, 4096, 7168, 128, 0, 1)])
def test_prepared_bytes(L, G, N, K, group, zeros, gated):
    """Whole blocks of 64 rows (a gated matrix: 32 of either projection) by 128 columns: codes, scales, zero points."""
    panels = -(-N // 2 // 32) if gated else -(-N // 64)
    want = G * panels * -(-K // 128) * (64 * 64 + 64 * (128 // group) * (3 if zeros else 2))
    assert L.nvfp4_w4_prepared_bytes(G, N, K, group, zeros, gated) == want
    for bad in [(0, N, K, group), (G, 0, K, group), (G, N, 0, group), (G, N, K + 4, group), (G, N, K, 48), (G, 1 << 24, K, group)]:
        assert L.nvfp4_w4_prepared_bytes(*bad, zeros, gated) == 0
    assert L.nvfp4_w4_prepared_bytes(1, 33, 128, 32, 0, 1) == 0


@pytest.mark.parametrize("M", [5, 40, 3000])
def test_linear(L, M):
    need = L.nvfp4_w4_linear_workspace_bytes(M, 4096, 4096, 64)
    assert (need > 0) == (M == 3000)
    if need:
        assert need >= 4096 * 4096 * 2 + 64 * 4096 * 4
    a = dict(x=P, dtype=BF, M=M, K=4096, ldx=4096, N=4096, w=1 << 32, group=64, zeros=0, y=1 << 34, ws=1 << 36, bytes=need, stream=None)
    for kw, st in [(dict(M=-1), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(dtype=F32), 1), (dict(group=100), 1), (dict(x=None), 1), (dict(w=None), 1),
                   (dict(y=None), 1), (dict(K=4092), 2), (dict(N=1 << 24), 2), (dict(M=1 << 24), 2), (dict(ldx=4088), 3), (dict(ldx=4100), 3),
                   (dict(x=P + 8), 3), (dict(w=(1 << 32) + 8), 3), (dict(y=(1 << 34) + 2), 3), (dict(ws=(1 << 36) + 16), 3)]:
        refuses(L, "nvfp4_w4_linear", changed(a, **kw), st)
    if need:
        refuses(L, "nvfp4_w4_linear", changed(a, bytes=need - 1), 4)
        refuses(L, "nvfp4_w4_linear", changed(a, ws=None), 1)
    for bad in [(-1, 64, 64, 32), (M, 0, 64, 32), (M, 64, 60, 32), (M, 64, 64, 16), (M, 1 << 24, 64, 32)]:
        assert L.nvfp4_w4_linear_workspace_bytes(*bad) == 0


def test_moe(L):
    need = L.nvfp4_w4_moe_workspace_bytes(5, 256, 128, 16, 4, 1)
    a = dict(x=P, dtype=BF, T=5, H=256, ldx=256, I=128, E=16, topk=4, router=2 * P, w13=1 << 30, w2=1 << 31, s13=1 << 32, s2=1 << 33, group=32,
             zeros=1, act=0, y=1 << 34, ws=1 << 35, bytes=need, stream=None)
    for kw, st in [(dict(T=-1), 1), (dict(H=0), 1), (dict(I=0), 1), (dict(E=0), 1), (dict(topk=0), 1), (dict(dtype=F32), 1), (dict(group=256), 1),
                   (dict(act=3), 1), (dict(act=-1), 1), (dict(x=None), 1), (dict(router=None), 1), (dict(w13=None), 1), (dict(w2=None), 1),
                   (dict(s13=None), 1), (dict(s2=None), 1), (dict(y=None), 1), (dict(ws=None), 1), (dict(H=252), 2), (dict(I=124), 2), (dict(T=65), 2),
                   (dict(topk=17), 2), (dict(E=3), 2), (dict(E=1025), 2), (dict(T=64, topk=9), 2), (dict(H=16392, ldx=16392), 2), (dict(I=16392), 2),
                   (dict(ldx=248), 3), (dict(ldx=260), 3), (dict(x=P + 8), 3), (dict(router=2 * P + 8), 3), (dict(w13=(1 << 30) + 8), 3),
                   (dict(s2=(1 << 33) + 4), 3), (dict(y=(1 << 34) + 2), 3), (dict(ws=(1 << 35) + 64), 3), (dict(bytes=need - 1), 4)]:
        refuses(L, "nvfp4_w4_moe", changed(a, **kw), st)


@pytest.mark.parametrize("T,H,I,E,topk,shared", [(0, 8, 8, 1, 1, 0), (1, 7168, 2048, 384, 8, 1), (64, 256, 64, 1024, 8, 1), (32, 16384, 16384, 16, 16, 0)])
def test_moe_workspace(L, T, H, I, E, topk, shared):
    rows = T * (topk + shared)
    n = L.nvfp4_w4_moe_workspace_bytes(T, H, I, E, topk, shared)
    parts = T * E * 4 + rows * I * 2 + rows * H * 4
    assert parts <= n <= parts + 16384 + 4 * (H // 64 + 1)
    for bad in [(65, H, I, E, topk), (-1, H, I, E, topk), (T, H + 4, I, E, topk), (T, H, I + 4, E, topk), (T, H, I, 1025, topk), (T, H, I, E, E + 1),
                (T, 16392, I, E, topk), (64, H, I, 1024, 16)]:
        assert L.nvfp4_w4_moe_workspace_bytes(*bad, shared) == 0


def test_residual_norm_fp8(L):
    a = dict(f=P, dtype=BF, r=2 * P, rd=F32, M=6, K=64, ldf=64, ldr=64, ga=3 * P, gate=4 * P, kind=1, groups=3, scale=1.0, gb=5 * P, eps=1e-6,
             ro=6 * P, q=7 * P, xs=8 * P, lds=8, y=9 * P, stats=None, stream=None)
    nan = float("nan")
    for kw, st in [(dict(rd=HF), 1), (dict(dtype=F32), 1), (dict(M=-1, lds=0), 1), (dict(f=None), 1), (dict(gate=None), 1), (dict(kind=0), 1),
                   (dict(eps=-1.0), 1), (dict(eps=nan), 1), (dict(scale=nan), 1), (dict(ro=None), 1), (dict(gb=None), 1), (dict(q=None), 1),
                   (dict(xs=None), 1), (dict(K=72, ldf=72, ldr=72), 2), (dict(K=16400, ldf=16400, ldr=16400), 2), (dict(groups=4), 2),
                   (dict(ldf=56), 3), (dict(ldr=68), 3), (dict(lds=4), 3), (dict(lds=10), 3), (dict(q=7 * P + 8), 3), (dict(xs=8 * P + 4), 3),
                   (dict(y=9 * P + 8), 3), (dict(ga=3 * P + 8), 3), (dict(rd=BF, ro=2 * P, stats=10 * P), 1), (dict(rd=BF, ro=2 * P, ldr=72), 3)]:
        refuses(L, "nvfp4_residual_norm_fp8", changed(a, **kw), st)


# every operand of a call in a range of its own: (arguments, bytes, written ones)
CALLS = {
    "nvfp4_w4_prepare": (dict(codes=0, scales=0, zeros=0, dtype=BF, G=2, N=70, K=264, group=64, gated=0, out=0, stream=None),
                         dict(codes=2 * 70 * 132, scales=2 * 70 * 5 * 2, zeros=2 * 70 * 5, out=2 * 2 * 3 * (4096 + 64 * 2 * 3)), ["out"]),
    "nvfp4_w4_linear": (dict(x=0, dtype=HF, M=5000, K=512, ldx=520, N=512, w=0, group=128, zeros=1, y=0, ws=0, bytes=1 << 20, stream=None),
                        dict(x=(4999 * 520 + 512) * 2, w=8 * 4 * (4096 + 64 * 3), y=5000 * 512 * 2, ws=512 * 512 * 2 + 4 * 512 * 4), ["y", "ws"]),
    "nvfp4_w4_moe": (dict(x=0, dtype=BF, T=5, H=256, ldx=264, I=128, E=4, topk=2, router=0, w13=0, w2=0, s13=0, s2=0, group=128, zeros=0, act=0,
                          y=0, ws=0, bytes=1 << 19, stream=None),
                     dict(x=(4 * 264 + 256) * 2, router=4 * 256 * 2, w13=4 * 4 * 2 * 4224, w2=4 * 4 * 4224, s13=4 * 2 * 4224, s2=4 * 4224,
                          y=5 * 256 * 2, ws=5 * 4 * 4 + 15 * 128 * 2 + 15 * 256 * 4), ["y", "ws"]),
    "nvfp4_residual_norm_fp8": (
        dict(f=0, dtype=BF, r=0, rd=F32, M=6, K=256, ldf=264, ldr=272, ga=0, gate=0, kind=1, groups=3, scale=1.0, gb=0, eps=1e-6, ro=0, q=0,
             xs=0, lds=8, y=0, stats=0, stream=None),
        dict(f=(5 * 264 + 256) * 2, r=(5 * 272 + 256) * 4, ga=512, gate=3 * 512, gb=512, ro=6 * 256 * 4, q=6 * 256, xs=(8 + 6) * 4, y=6 * 256 * 2,
             stats=6 * 8), ["ro", "q", "xs", "y", "stats"]),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_nothing_written_overlaps_another_operand(L, name):
    base, sizes, written = CALLS[name]
    at = {o: (1 << 26) + (i << 24) for i, o in enumerate(sizes)}
    base = {**base, **at}
    if not torch.cuda.is_available():  # the pointers are not real: the call ends at the device
        assert getattr(L, name)(*changed(base)) in NO_DEVICE
    for w in written:
        for o, n in sizes.items():
            if o == w:
                continue
            for p in (at[o], at[o] + (n - 1) // 256 * 256, at[o] - (sizes[w] - 1) // 256 * 256):
                if (w, o) == ("ro", "r") and p == at["r"]:
                    continue  # in place: rules of its own
                refuses(L, name, changed(base, **{w: p}), 1)
                assert b"overlap" in L.nvfp4_last_error_string(), (w, o)


def test_valid_calls_without_a_gpu_fail_cleanly(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for name, (base, sizes, _) in CALLS.items():
        at = {o: (1 << 26) + (i << 24) for i, o in enumerate(sizes)}
        assert getattr(L, name)(*changed({**base, **at})) in NO_DEVICE
    assert L.nvfp4_w4_linear(None, BF, 0, 64, 64, 64, P, 32, 0, None, None, 0, None) in NO_DEVICE
    assert L.nvfp4_w4_moe(None, BF, 0, 64, 64, 64, 4, 2, P, P, P, None, None, 32, 0, 0, None, 2 * P, 1 << 20, None) in NO_DEVICE


# ---------------------------------------------------------------- the torch layer

def fake(G, N, K, group=128, dtype=torch.bfloat16, zeros=False, gated=False):
    return ops.W4Weight(torch.zeros(16, dtype=torch.uint8), G, N, K, group, dtype, zeros, gated)


def test_torch_layer_refuses_cpu_tensors():
    x, codes = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(16, 32, dtype=torch.uint8)
    for f in [lambda: ops.w4_prepare(codes, torch.zeros(16, 1, dtype=torch.bfloat16)), lambda: ops.w4_linear(x, fake(1, 16, 64)),
              lambda: ops.w4_moe(x, torch.zeros(2, 64, dtype=torch.bfloat16), fake(2, 64, 64, gated=True), fake(2, 64, 32), 1),
              lambda: ops.residual_norm_fp8(x, x, x[0])]:
        with pytest.raises(ValueError, match="CUDA"):
            f()


@pytest.mark.parametrize("other", [dict(G=2), dict(N=65), dict(K=72), dict(gated=True)])
def test_weights_of_other_sizes(other):
    w = dataclasses.replace(fake(1, 64, 64), **other)
    with pytest.raises(ValueError, match="expected"):
        ops._w4(w, "w", 1, 64, 64, False)


@pytest.mark.parametrize("other", [dict(dtype=torch.float16), dict(group=64), dict(has_zeros=True)])
def test_weights_of_other_kinds(other):
    w = dataclasses.replace(fake(1, 64, 64), **other)
    ops._w4(w, "w", 1, 64, 64, False)
    with pytest.raises(ValueError, match="those of the other weights"):
        ops._w4(w, "w", 1, 64, 64, False, fake(1, 64, 64))


def test_weights_whose_data_do_not_fit(L):
    """A weight built by hand: too few bytes, too many, another type, every other byte."""
    n = L.nvfp4_w4_prepared_bytes(1, 64, 64, 128, 0, 0)
    for data in (torch.zeros(n - 1, dtype=torch.uint8), torch.zeros(n + 1, dtype=torch.uint8), torch.zeros(n, dtype=torch.int8),
                 torch.zeros(2 * n, dtype=torch.uint8)[::2], torch.zeros(0, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="are not the data of"):
            ops._w4_whole(dataclasses.replace(fake(1, 64, 64), data=data), "w", 1, 64, 64, False)
    ops._w4_whole(dataclasses.replace(fake(1, 64, 64), data=torch.zeros(n, dtype=torch.uint8)), "w", 1, 64, 64, False)


def test_workspace_of_unsupported_sizes():
    with pytest.raises(ValueError, match="unsupported"):
        ops.w4_moe_workspace(65, 64, 64, 8, 2, False, "cpu")


# ---------------------------------------------------------------- arithmetic

def test_codes_as_subnormals():
    """The bits of c in the low or high half of a byte are, as a bf16 or fp16 number, c or 16 c times its smallest
    subnormal, and taking z off by a multiplication and addition of that type is exact."""
    c = torch.arange(16)
    for dt, step, up in ((torch.bfloat16, -133, 126), (torch.float16, -24, 14)):
        for shift in (0, 4):
            v = (c << shift).to(torch.int16).view(dt).double()
            assert torch.equal(v, c.double() * 2.0 ** (step + shift))
            for z in range(16):
                d = v * 2.0 ** (up - shift) - z * 2.0 ** (step + up)
                assert torch.equal(d.to(dt).double(), d) and torch.equal(d, (c - z).double() * 2.0 ** (step + up))


@pytest.mark.parametrize("dt,top,most,bias,mantissa", [(torch.bfloat16, 60, 126, 127, 7), (torch.float16, 14, 15, 15, 10)])
def test_powers_of_two_of_rows(dt, top, most, bias, mantissa):
    """For every largest magnitude of a row: both factors are numbers of the type, the row stays finite, and bf16 loses nothing of
    elements down to 2^-150 of it, fp16 nothing above 2^-36 of it."""
    bits = torch.arange(1, (2 << (15 - mantissa - 1) << mantissa) - 0, dtype=torch.int32)
    values = bits.to(torch.int16).view(dt)
    bits, values = bits[torch.isfinite(values)], values[torch.isfinite(values)].double()
    power = torch.clamp(top - ((bits >> mantissa) - bias), max=most)
    low = ((power + bias) << mantissa).to(torch.int16).view(dt).double()
    high = ((power + bias - 4) << mantissa).to(torch.int16).view(dt).double()
    assert torch.equal(low, 2.0 ** power.double()) and torch.equal(high, low / 16)
    scaled = values * low
    assert (scaled < 2.0 ** (top + 1)).all()
    assert torch.equal(scaled.to(dt).double(), scaled)  # the largest itself
    off = ((values * high).to(dt).double() - values * high).abs() * 16 / low
    assert (off <= 2.0 ** -37 * values).all() if dt == torch.float16 else (off == 0).all()


def test_scale_of_every_fp32_mantissa():
    """fl32(m / 448) from the product with fl32(1 / 448), corrected once by its remainder (exact in fp32), for every mantissa."""
    m = (np.arange(2 ** 23, dtype=np.uint32) | np.uint32(0x3F800000)).view(np.float32).astype(np.float64)
    r = float(np.float32(1 / 448.0))
    f32 = lambda v: v.astype(np.float32).astype(np.float64)  # noqa: E731
    q = f32(m * r)
    rest = m - q * 448.0
    assert np.array_equal(f32(rest), rest)
    exact = q + rest * r  # float64's own rounding is far from the midpoints of two fp32 values
    got = f32(exact)
    assert (np.abs(np.abs(exact - got) / np.spacing(got.astype(np.float32)) - 0.5) > 0.01).all()
    assert np.array_equal(got, f32(m / 448.0))


@pytest.mark.parametrize("topk", range(1, 17))
def test_token_of_an_entry(topk):
    """entry / topk by a product with ceil(2^16 / topk), for every entry."""
    inverse = (65536 + topk - 1) // topk
    assert all(((f * inverse) >> 16) == f // topk for f in range(512))
