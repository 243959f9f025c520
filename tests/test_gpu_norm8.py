"""The residual norm with an 8-bit output: the sum, the 16-bit output and the statistics bit for bit those of the residual
norm, the codes and scales against the definition in 64 bits, and as the 8-bit product's operand."""

import pytest
import torch

from nvfp4_block_scaled_quant_gb300 import ops

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def make(M, K, kind, rkind, gate, after, seed=0):
    g = torch.Generator(device="cuda").manual_seed(31 * seed + M + K)
    dt = TYPES[kind]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    shape = {"none": None, "channel": (K,), "row": (M, 1), "groups": (2, K)}[gate]
    return dict(f=(normal(M, K) * 3).to(dt), r=(normal(M, K) * torch.exp(0.5 * normal(K))).to(TYPES[rkind]),
                gamma_after=(1 + 0.1 * normal(K)).to(dt) if after else None, gate=None if shape is None else (0.5 * normal(*shape)).to(dt),
                scale=0.5, gamma_before=(1 + 0.1 * normal(K)).to(dt))


def y64(a, eps=1e-6):
    M, K = a["f"].shape
    f, r = a["f"].double(), a["r"].double()
    if a["gamma_after"] is not None:
        f = f * (f.square().mean(1, keepdim=True) + eps).rsqrt() * a["gamma_after"].double()
    if a["gate"] is not None:
        gate = a["gate"].double()
        gate = gate.expand(M, K) if gate.dim() == 1 or gate.shape == (M, 1) else gate.repeat_interleave(M // gate.shape[0], 0)
        f = f * gate
    ro = r + a["scale"] * f
    return ro * (ro.square().mean(1, keepdim=True) + eps).rsqrt() * a["gamma_before"].double()


def verify(a, eps=1e-6):
    M, K = a["f"].shape
    r_out, q, s, y, stats = ops.residual_norm_fp8(**a, eps=eps, want_y=True, save=True)
    ref = ops.residual_norm(**a, eps=eps, save=True)
    assert torch.equal(r_out, ref[0]) and torch.equal(y, ref[1]) and torch.equal(stats, ref[2])
    plain = ops.residual_norm_fp8(**a, eps=eps)
    assert torch.equal(plain[0], r_out) and torch.equal(plain[1].view(torch.uint8), q.view(torch.uint8)) and torch.equal(plain[2], s)
    assert plain[3] is None and s.shape == ((K + 127) // 128, M) and q.dtype == torch.float8_e4m3fn
    want = y64(a, eps)
    # fp32 arithmetic of y: the two statistics (a mean of K squares in a tree of sums, half of its error each), about
    # ten products and sums; the sum's cancellation counts against |r| + |scale gate n|
    rel = 2.0 ** -18
    size = want.abs() + rel * want.abs().amax(dim=1, keepdim=True)
    yb = torch.nn.functional.pad(want, (0, -K % 128)).view(M, -1, 128)
    top = yb.abs().amax(dim=2)
    floor = want.abs().amax(dim=1, keepdim=True)
    assert ((s.T.double() - top / 448).abs() <= rel * (top + floor) / 448).all()
    sc = s.T.double().repeat_interleave(128, dim=1)[:, :K]
    got = q.double() * sc
    # half a step of e4m3: 2^-4 of the value, 2^-10 of the scale among the smallest
    bound = torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * sc) + rel * (size + floor)
    assert ((got - want).abs() <= bound).all()
    return q, s, want


@pytest.mark.parametrize("kind,rkind", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp32"), ("fp16", "fp32")])
@pytest.mark.parametrize("gate", ["none", "channel", "row", "groups"])
@pytest.mark.parametrize("M,K,after", [(2, 256, True), (6, 1552, False), (400, 1040, True), (700, 128, False)])
def test_against_definition(M, K, after, gate, kind, rkind):
    verify(make(M, K, kind, rkind, gate, after))


@pytest.mark.parametrize("M,K", [(1, 16), (1, 7168), (5, 144), (3, 16384), (305, 16), (306, 112), (330, 7168), (310, 16384), (1000, 8192), (4, 8208)])
def test_widths(M, K):
    verify(make(M, K, "bf16", "fp32", "channel", True, 1))


@pytest.mark.parametrize("M", [3, 500])
def test_blocks_of_zeros_and_bad_values(M):
    a = make(M, 512, "bf16", "bf16", "none", False, 2)
    a["f"][:, 128:256] = 0
    a["r"][:, 128:256] = 0
    q, s, _ = verify(a)
    assert (s[1] == 0).all() and (q[:, 128:256].view(torch.uint8) == 0).all()
    ref = [t.clone() for t in (q.view(torch.uint8), s)]
    a["r"][M - 1, 300] = float("nan")
    a["f"][0, 10] = float("inf")
    _, q, s, _ = ops.residual_norm_fp8(**a)
    assert torch.isnan(s[:, M - 1]).all() and not torch.isfinite(s[0, 0])
    assert torch.equal(q[1:M - 1].view(torch.uint8), ref[0][1:M - 1]) and torch.equal(s[:, 1:M - 1], ref[1][:, 1:M - 1])


@pytest.mark.parametrize("M", [2, 400])
def test_tiny_and_large_rows(M):
    """Rows from 1e-30 to 1e15: the codes of the same row at another size are the same where eps vanishes."""
    a = make(M, 640, "bf16", "fp32", "none", False, 3)
    for size in (1e-16, 1e-6, 1e15):
        b = dict(a, f=torch.zeros_like(a["f"]), r=a["r"] * size)
        verify(b, eps=0.0)
    b = dict(a, f=torch.zeros_like(a["f"]), r=a["r"] * 1e-30, gamma_before=a["gamma_before"] * 1e-4)
    verify(b, eps=1e-6)


def test_strides_in_place_and_no_rows():
    a = make(40, 272, "fp16", "fp16", "row", True, 4)
    want = ops.residual_norm_fp8(**a)
    wide = torch.full((40, 400), float("nan"), device="cuda", dtype=torch.float16)
    wide[:, 64:336] = a["f"]
    rw = torch.full((40, 320), float("nan"), device="cuda", dtype=torch.float16)
    rw[:, 8:280] = a["r"]
    got = ops.residual_norm_fp8(**dict(a, f=wide[:, 64:336], r=rw[:, 8:280]))
    for u, v in zip(got[:3], want[:3]):
        assert torch.equal(u.view(torch.uint8) if u.dtype == torch.float8_e4m3fn else u, v.view(torch.uint8) if v.dtype == torch.float8_e4m3fn else v)
    r = a["r"].clone()
    got = ops.residual_norm_fp8(**dict(a, r=r), out=r)
    assert got[0] is r and torch.equal(r, want[0]) and torch.equal(got[2], want[2])
    empty = ops.residual_norm_fp8(**dict(a, f=a["f"][:0], r=a["r"][:0], gate=a["gate"][:0]))
    assert empty[0].shape == (0, 272) and empty[1].shape == (0, 272) and empty[2].shape == (3, 0)


@pytest.mark.parametrize("M", [1, 7, 400])
def test_feeds_the_product(M):
    """The 8-bit product takes the output as it is: equal to the product of the values it stands for."""
    K, N = 656, 200
    a = make(M, K, "bf16", "bf16", "channel", True, 5)
    _, q, s, _ = ops.residual_norm_fp8(**a)
    w = (torch.randn(N, K, device="cuda", generator=torch.Generator(device="cuda").manual_seed(9)) * K ** -0.5).bfloat16()
    wq, ws = ops.fp8_quantize_weight(w)
    y = ops.fp8_gemm(q, s, wq, ws)
    deq = q.double() * s.T.double().repeat_interleave(128, dim=1)[:, :K]
    wd = wq.double() * ws.double().repeat_interleave(128, dim=0)[:N].repeat_interleave(128, dim=1)[:, :K]
    want = deq @ wd.T
    err = 2.0 ** -23 * (K / 32 + 16) * (deq.abs() @ wd.abs().T)
    assert ((y.double() - want).abs() <= err + 2.0 ** -8 * (want.abs() + err)).all()
    # and close to the quantiser's on the rounded output, up to the second rounding
    _, y16 = ops.residual_norm(**a)
    other = ops.fp8_linear(y16, wq, ws)
    assert (y.double() - other.double()).norm() <= 2.0 ** -4 * other.double().norm()


def test_gradients_of_the_kept_statistics():
    """A training step that quantises behind the norm: the residual norm's backward with these statistics."""
    a = make(30, 256, "bf16", "fp32", "row", True, 6)
    g = torch.Generator(device="cuda").manual_seed(3)
    dr, dy = torch.randn(30, 256, generator=g, device="cuda"), torch.randn(30, 256, generator=g, device="cuda").bfloat16()
    kw = {k: a[k] for k in ("gamma_after", "gate", "scale", "gamma_before")}
    got = ops.residual_norm_backward(dr, dy, a["f"], a["r"], ops.residual_norm_fp8(**a, save=True)[4], **kw)
    want = ops.residual_norm_backward(dr, dy, a["f"], a["r"], ops.residual_norm(**a, save=True)[2], **kw)
    assert all(torch.equal(u, v) for u, v in zip(got, want))


@pytest.mark.parametrize("M", [4, 500])
def test_graph(M):
    a = make(M, 384, "bf16", "bf16", "none", True, 7)
    want = ops.residual_norm_fp8(**a, want_y=True)
    static = dict(a, f=a["f"].clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ops.residual_norm_fp8(**static, want_y=True)
    static["f"].zero_()
    graph.replay()
    static["f"].copy_(a["f"])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1].view(torch.uint8), want[1].view(torch.uint8)) and torch.equal(got[2], want[2])
