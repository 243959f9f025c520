"""FP8 block-scaled linear on the GPU against its definition in 64 bits.

Exact cases use small integer codes and power-of-two scales, so every product and partial sum is
exact in fp32 whatever the order, and the output is the correctly rounded exact value: any index,
scale or layout mistake shows.  Random cases are held to a bound: half a step of the output type,
plus one fp32 step of the sum of absolute products for each of the additions an output can pass
through (128 inside a K block, one per block, at most 8 split partial sums, 4 for the scales).
"""

import pytest
import torch

from nvfp4_block_scaled_quant_gb300 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn


def quantize_ref(x, rows):
    """Codes as float64 values and fp32 scales of (R, K) blocks of `rows` x 128, from the definition."""
    R, K = x.shape
    q = torch.zeros(R, K, dtype=torch.float64, device=x.device)
    s = torch.zeros((R + rows - 1) // rows, (K + 127) // 128, dtype=torch.float32, device=x.device)
    for i in range(s.shape[0]):
        for b in range(s.shape[1]):
            blk = x[i * rows:(i + 1) * rows, b * 128:(b + 1) * 128].double()
            sc = (blk.abs().max() / 448.0).float()
            s[i, b] = sc
            if sc > 0:
                v = (blk / sc.double()).float()  # the correctly rounded fp32 quotient
                q[i * rows:(i + 1) * rows, b * 128:(b + 1) * 128] = v.clamp(-448, 448).to(F8).double()
    return q, s


def product_ref(q, s, w, ws):
    """(y, sum of absolute products) in float64; q, w values, s (M, KB), ws (NB, KB)."""
    K, N = q.shape[1], w.shape[0]
    y = torch.zeros(q.shape[0], N, dtype=torch.float64, device=q.device)
    a = torch.zeros_like(y)
    for b in range(0, K, 128):
        f = s[:, b // 128:b // 128 + 1].double() * ws[:, b // 128].double().repeat_interleave(128)[:N]
        y += (q[:, b:b + 128] @ w[:, b:b + 128].T) * f
        a += (q[:, b:b + 128].abs() @ w[:, b:b + 128].abs().T) * f
    return y, a


def assert_close(y, ref, mag, K):
    u = torch.finfo(y.dtype).eps / 2
    bound = u * ref.abs() + torch.finfo(y.dtype).smallest_normal * u + (128 + (K + 127) // 128 + 8 + 4) * 2.0 ** -23 * mag * (1 + u)
    err = (y.double() - ref).abs()
    assert torch.isfinite(y).all()
    assert (err <= bound).all(), f"worst excess {(err - bound).max().item()} at {(err - bound).argmax().item()}"


def integer_case(M, K, N, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.randint(-3, 4, (M, K), generator=g, device=DEV).float()
    w = torch.randint(-3, 4, (N, K), generator=g, device=DEV).float()
    KB, NB = (K + 127) // 128, (N + 127) // 128
    s = torch.exp2(torch.randint(-2, 3, (M, KB), generator=g, device=DEV).float())
    ws = torch.exp2(torch.randint(-2, 3, (NB, KB), generator=g, device=DEV).float())
    return q, w, s, ws


def padded_scales(s):
    M, KB = s.shape
    buf = torch.full((KB, (M + 3) // 4 * 4), float("nan"), dtype=torch.float32, device=DEV)
    buf[:, :M] = s.T
    return buf[:, :M]


SHAPES = [(1, 128, 128), (1, 16, 1), (2, 144, 129), (5, 1000 // 16 * 16, 77), (16, 512, 256), (17, 1536, 300), (33, 2000, 130),
          (64, 640, 512), (65, 7168, 136), (128, 256, 1000), (129, 272, 257), (200, 1040, 520), (256, 128, 384),
          (257, 128, 256), (300, 2000, 1137), (512, 896, 512), (777, 1552, 1025), (2100, 256, 264)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_gemm_exact_integers(M, K, N, dtype):
    q, w, s, ws = integer_case(M, K, N, seed=M + K + N)
    y = ops.fp8_gemm(q.to(F8), padded_scales(s), w.to(F8), ws, dtype=dtype)
    ref, mag = product_ref(q.double(), s, w.double(), ws)
    assert mag.max() * 16 < 2 ** 24  # multiples of 2^-4 below 2^20: every partial sum is exact in fp32
    assert torch.equal(y, ref.to(dtype))
    assert ops.device_error() == (0, 0)


@pytest.mark.parametrize("M,K", [(1, 16), (1, 7168), (3, 144), (17, 2000), (130, 640), (1000, 272)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_quantize_act_matches_definition(M, K, dtype):
    g = torch.Generator(device=DEV).manual_seed(M * K)
    x = (torch.randn(M, K, generator=g, device=DEV) * torch.exp(2 * torch.randn(M, 1, generator=g, device=DEV))).to(dtype)
    if M > 2:
        x[1, :min(K, 128)] = 0  # an all-zero block
        x[2] = 2.0 ** -24 if dtype == torch.float16 else 2.0 ** -133  # subnormal values
    q, s = ops.fp8_quantize_act(x)
    rq, rs = quantize_ref(x, 1)
    assert q.dtype == F8 and s.shape == (rs.shape[1], M)
    assert torch.equal(s.T, rs)
    assert torch.equal(q.double(), rq)


@pytest.mark.parametrize("N,K", [(1, 16), (128, 128), (130, 272), (300, 1536)])
def test_quantize_weight_matches_definition(N, K):
    g = torch.Generator(device=DEV).manual_seed(N * K)
    for dtype in (torch.bfloat16, torch.float16):
        w = torch.randn(N, K, generator=g, device=DEV).to(dtype)
        q, s = ops.fp8_quantize_weight(w)
        rq, rs = quantize_ref(w, 128)
        assert torch.equal(s, rs) and torch.equal(q.double(), rq)


@pytest.mark.parametrize("M,K,N", [(1, 7168, 256), (7, 1536, 1000), (2, 16, 3), (16, 656, 130), (17, 2000, 77), (32, 1024, 8448),
                                   (33, 1024, 260), (37, 1536, 640), (24, 7168, 2700),
                                   (48, 2000, 1136), (64, 512, 500), (64, 4096, 130), (129, 1024, 129), (300, 2000, 400)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_linear_random(M, K, N, dtype):
    g = torch.Generator(device=DEV).manual_seed(M + K)
    x = (torch.randn(M, K, generator=g, device=DEV) * torch.exp(0.7 * torch.randn(K, generator=g, device=DEV))).to(dtype)
    w, ws = ops.fp8_quantize_weight((torch.randn(N, K, generator=g, device=DEV) * K ** -0.5).to(dtype))
    y = ops.fp8_linear(x, w, ws)
    q, s = quantize_ref(x, 1)
    ref, mag = product_ref(q, s, w.double(), ws)
    assert_close(y, ref, mag, K)
    # the two calls give the one call's bits, also on the codes as raw bytes
    xq, xs = ops.fp8_quantize_act(x)
    assert torch.equal(y, ops.fp8_gemm(xq.view(torch.uint8), xs, w.view(torch.uint8), ws, dtype=dtype))


def test_repeated_calls_give_the_same_bits():
    g = torch.Generator(device=DEV).manual_seed(3)
    for M in (1, 40, 300):
        x = torch.randn(M, 2048, generator=g, device=DEV).bfloat16()
        w, ws = ops.fp8_quantize_weight(torch.randn(777, 2048, generator=g, device=DEV).bfloat16())
        y = ops.fp8_linear(x, w, ws)
        for _ in range(3):
            assert torch.equal(y, ops.fp8_linear(x, w, ws))


@pytest.mark.parametrize("M", [3, 40, 300])
def test_nan_and_inf_stay_in_their_rows(M):
    g = torch.Generator(device=DEV).manual_seed(M)
    x = torch.randn(M, 512, generator=g, device=DEV).bfloat16()
    w, ws = ops.fp8_quantize_weight(torch.randn(256, 512, generator=g, device=DEV).bfloat16())
    clean = ops.fp8_linear(x, w, ws)
    x[0, 200] = float("nan")
    x[2, 300] = float("inf")
    y = ops.fp8_linear(x, w, ws)
    assert torch.isnan(y[0]).all() and torch.isnan(y[2]).all()
    keep = [i for i in range(M) if i not in (0, 2)]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("M", [5, 50, 300])
def test_strided_rows_and_given_buffers(M):
    g = torch.Generator(device=DEV).manual_seed(M)
    big = torch.randn(M, 1024 + 16, generator=g, device=DEV).bfloat16()
    x = big[:, 8:8 + 512]
    w, ws = ops.fp8_quantize_weight(torch.randn(200, 512, generator=g, device=DEV).bfloat16())
    ref = ops.fp8_linear(x.contiguous(), w, ws)
    out = torch.full((M + 1, 200), 7.0, dtype=torch.bfloat16, device=DEV)
    work = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    y = ops.fp8_linear(x, w, ws, out=out[:M], workspace=work)
    assert torch.equal(y, ref) and y.data_ptr() == out.data_ptr()
    assert (out[M] == 7.0).all()  # the row behind the last is left as it was
    assert torch.equal(big[:, 8:520], x)


def test_no_rows():
    w, ws = ops.fp8_quantize_weight(torch.randn(8, 32, device=DEV).bfloat16())
    assert ops.fp8_linear(torch.empty(0, 32, dtype=torch.bfloat16, device=DEV), w, ws).shape == (0, 8)


@pytest.mark.parametrize("M", [1, 300])
def test_captured_and_on_another_stream(M):
    g = torch.Generator(device=DEV).manual_seed(M)
    x = torch.randn(M, 1536, generator=g, device=DEV).bfloat16()
    w, ws = ops.fp8_quantize_weight(torch.randn(512, 1536, generator=g, device=DEV).bfloat16())
    ref = ops.fp8_linear(x, w, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = ops.fp8_linear(x, w, ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ops.fp8_linear(x, w, ws)
    x2 = torch.randn(M, 1536, generator=g, device=DEV).bfloat16()
    ref2 = ops.fp8_linear(x2, w, ws)
    x.copy_(x2)
    graph.replay()
    assert torch.equal(y, ref2)


def test_refusals():
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device=DEV)
    w, ws = ops.fp8_quantize_weight(torch.ones(64, 256, dtype=torch.bfloat16, device=DEV))
    xq, xs = ops.fp8_quantize_act(x)
    bad = [lambda: ops.fp8_linear(x.float(), w, ws), lambda: ops.fp8_linear(x[:, :128], w, ws),
           lambda: ops.fp8_linear(x, w, ws.T.contiguous()), lambda: ops.fp8_linear(x, w.float(), ws),
           lambda: ops.fp8_linear(x.cpu(), w, ws), lambda: ops.fp8_linear(x.T, w, ws),
           lambda: ops.fp8_gemm(xq, xs[:, :3], w, ws), lambda: ops.fp8_gemm(xq, xs.double(), w, ws),
           lambda: ops.fp8_gemm(xq, xs, w, ws, dtype=torch.float32),
           lambda: ops.fp8_linear(x, w, ws, out=torch.empty(4, 65, dtype=torch.bfloat16, device=DEV)),
           lambda: ops.fp8_gemm(ops.fp8_quantize_act(x[:3])[0], torch.zeros(2, 3, device=DEV), w, ws)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in [lambda: ops.fp8_linear(x.repeat(16, 1), w, ws, workspace=torch.empty(256, dtype=torch.uint8, device=DEV)),
              lambda: ops.fp8_quantize_act(torch.zeros(4, 24, dtype=torch.bfloat16, device=DEV)),
              lambda: ops.fp8_quantize_act(torch.zeros(4, 36, dtype=torch.bfloat16, device=DEV)[:, :32]),
              lambda: ops.fp8_quantize_act(torch.zeros(1, 32, dtype=torch.bfloat16, device=DEV).expand(4, 32))]:
        with pytest.raises(RuntimeError, match="nvfp4 status"):
            f()
