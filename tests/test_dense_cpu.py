"""CPU checks of the dense feed-forward operators: the C ABI refuses bad arguments on the host, before any
device is touched, with the right status and a message; workspace sizes; the torch layer's refusals."""

import ctypes

import pytest
import torch

from nvfp4_block_scaled_quant_gb300 import _lib, ops
from nvfp4_block_scaled_quant_gb300 import build as B

P = 1 << 20  # an aligned address that is never used: validation fails first
BF, HF, F32 = _lib.DT_BF16, _lib.DT_FP16, _lib.DT_FP32


@pytest.fixture(scope="module")
def L():
    B.build()
    return _lib.lib()


def refuses(L, name, args, want):
    assert getattr(L, name)(*args) == want, (name, args, L.nvfp4_last_error_string())
    assert L.nvfp4_last_error_string().startswith(name.encode())


def changed(base, **kw):
    """`base` (a dict in the order of the call's arguments) with some arguments replaced."""
    return tuple({**base, **kw}.values())


def test_fp8_quantisers(L):
    a = dict(x=P, dtype=BF, M=4, K=256, ldx=256, q=P, xs=P, lds=4, stream=None)
    for kw, st in [(dict(dtype=F32), 1), (dict(dtype=7), 1), (dict(M=-1), 1), (dict(K=0), 1), (dict(x=None), 1),
                   (dict(q=None), 1), (dict(xs=None), 1), (dict(K=264), 2), (dict(K=1 << 24, ldx=1 << 24), 2),
                   (dict(ldx=248), 3), (dict(ldx=260), 3), (dict(x=P + 2), 3), (dict(q=P + 8), 3), (dict(lds=3), 3), (dict(lds=6), 3)]:
        refuses(L, "nvfp4_fp8_quantize_act", changed(a, **kw), st)
    w = dict(w=P, dtype=HF, N=4, K=256, ldw=256, q=P, s=P, stream=None)
    for kw, st in [(dict(N=0), 1), (dict(dtype=F32), 1), (dict(q=None), 1), (dict(K=24, ldw=24), 2), (dict(ldw=16), 3), (dict(w=P + 4), 3)]:
        refuses(L, "nvfp4_fp8_quantize_weight", changed(w, **kw), st)


def test_fp8_gemm_and_linear(L):
    a = dict(xq=P, xs=P, lds=4, M=4, K=256, N=100, w=P, ws=P, dtype=BF, y=P, stream=None)
    for kw, st in [(dict(N=0), 1), (dict(dtype=F32), 1), (dict(w=None), 1), (dict(y=None), 1), (dict(xs=None), 1), (dict(K=250), 2),
                   (dict(N=1 << 24), 2), (dict(lds=2), 3), (dict(lds=5), 3), (dict(w=P + 8), 3), (dict(y=P + 2), 3)]:
        refuses(L, "nvfp4_fp8_gemm", changed(a, **kw), st)
    need = L.nvfp4_fp8_linear_workspace_bytes(100, 256)
    assert need >= 100 * 256 + 2 * 100 * 4 and L.nvfp4_fp8_linear_workspace_bytes(16, 256) == 0
    assert L.nvfp4_fp8_linear_workspace_bytes(100, 250) == 0 and L.nvfp4_fp8_linear_workspace_bytes(-1, 256) == 0
    b = dict(x=P, dtype=BF, M=100, K=256, ldx=256, N=100, w=P, ws=P, y=P, work=P, bytes=need, stream=None)
    for kw, st in [(dict(bytes=need - 1), 4), (dict(work=None), 1), (dict(work=P + 16), 3), (dict(N=-5), 1), (dict(w=None), 1),
                   (dict(y=None), 1), (dict(x=P + 8), 3), (dict(K=255), 2)]:
        refuses(L, "nvfp4_fp8_linear", changed(b, **kw), st)


def test_gated_linear(L):
    a = dict(x=P, dtype=BF, T=4, H=64, ldx=64, I=16, wg=P, wu=P, act=0, h=P, gu=None, stream=None)
    for kw, st in [(dict(act=3), 1), (dict(act=-1), 1), (dict(dtype=F32), 1), (dict(T=-1), 1), (dict(wg=None), 1), (dict(h=None), 1),
                   (dict(H=60, ldx=64), 2), (dict(I=12), 2), (dict(I=1 << 23), 2), (dict(ldx=56), 3), (dict(ldx=68), 3),
                   (dict(wu=P + 8), 3), (dict(gu=P + 8), 3)]:
        refuses(L, "nvfp4_gated_linear", changed(a, **kw), st)
    need = L.nvfp4_gated_linear_backward_workspace_bytes(4, 16)
    assert need == 256 and L.nvfp4_gated_linear_backward_workspace_bytes(4, 12) == 0
    b = dict(dh=P, lddh=16, x=P, ldx=64, dtype=BF, T=4, H=64, I=16, wg=P, wu=P, act=0, gu=P, dx=P, dwg=P, dwu=P, ws=P, bytes=need,
             stream=None)
    for kw, st in [(dict(gu=None), 1), (dict(dh=None), 1), (dict(dwu=None), 1), (dict(dwg=None), 1), (dict(bytes=0), 4),
                   (dict(lddh=8), 3), (dict(lddh=18), 3), (dict(dx=P + 2), 3), (dict(act=9), 1)]:
        refuses(L, "nvfp4_gated_linear_backward", changed(b, **kw), st)


def test_residual_norm(L):
    a = dict(f=P, dtype=BF, r=P, rd=F32, M=6, K=64, ldf=64, ldr=64, ga=P, gate=P, kind=1, groups=3, scale=1.0, gb=P, eps=1e-6, ro=P, y=P,
             stats=None, stream=None)
    nan = float("nan")
    for kw, st in [(dict(rd=HF), 1), (dict(dtype=F32), 1), (dict(M=-1), 1), (dict(f=None), 1), (dict(gate=None), 1), (dict(kind=0), 1),
                   (dict(kind=5), 1), (dict(eps=-1.0), 1), (dict(eps=nan), 1), (dict(scale=nan), 1), (dict(ro=None), 1), (dict(y=None), 1),
                   (dict(gb=None), 1), (dict(K=60), 2), (dict(K=16392, ldf=16392, ldr=16392), 2), (dict(groups=4), 2), (dict(groups=0), 2),
                   (dict(ldf=56), 3), (dict(ldr=68), 3), (dict(ga=P + 8), 3), (dict(gate=P + 2), 3), (dict(y=P + 8), 3),
                   (dict(ro=P, ldr=72), 3)]:
        refuses(L, "nvfp4_residual_norm", changed(a, **kw), st)
    need = L.nvfp4_residual_norm_backward_workspace_bytes(6, 64, 3, F32)
    assert need > 0 and L.nvfp4_residual_norm_backward_workspace_bytes(6, 64, 4, F32) == 0
    assert L.nvfp4_residual_norm_backward_workspace_bytes(0, 64, 1, F32) == 0
    b = dict(dro=P, lddr=64, dy=P, lddy=64, f=P, dtype=BF, r=P, rd=F32, M=6, K=64, ldf=64, ldr=64, stats=P, ga=P, gate=P, kind=1, groups=3,
             scale=1.0, gb=P, df=P, dr=P, dga=P, dgate=P, dgb=P, ws=P, bytes=need, stream=None)
    for kw, st in [(dict(stats=None), 1), (dict(df=None), 1), (dict(gb=None), 1), (dict(ga=None), 1), (dict(gate=None, kind=0), 1),
                   (dict(bytes=need - 1), 4), (dict(lddr=56), 3), (dict(lddy=66), 3), (dict(df=P + 8), 3), (dict(dga=P + 4), 3)]:
        refuses(L, "nvfp4_residual_norm_backward", changed(b, **kw), st)


def test_an_output_inside_an_input_is_refused(L):
    """Other blocks may still read what one writes; r_out at r's own address is the exception."""
    for y in (P, P + 512 * 3, P - 16):
        refuses(L, "nvfp4_fp8_linear", (P, BF, 4, 256, 256, 8, P, P, y, None, 0, None), 1)
        refuses(L, "nvfp4_gated_linear", (P, BF, 4, 256, 256, 8, P, P, 0, y, None, None), 1)
    refuses(L, "nvfp4_fp8_gemm", (P, P, 4, 4, 256, 8, P, P, BF, P + 1008, None), 1)
    far = 1 << 30
    for f, r, ro in [(P, far, P), (far, P, P + 128), (far, P, P - 128), (P, far, P + 4 * 128 - 16)]:
        refuses(L, "nvfp4_residual_norm", (f, BF, r, BF, 4, 64, 64, 64, None, None, 0, 0, 1.0, None, 1e-6, ro, None, None, None), 1)


@pytest.mark.parametrize("M,K,groups,kind", [(1, 8, 1, BF), (4096, 7168, 1, BF), (8192, 7168, 8, BF), (1001, 1544, 1, F32), (600, 64, 600, F32),
                                             (3, 16384, 3, F32), (100000, 256, 4, BF)])
def test_norm_workspace_holds_the_partial_sums(L, M, K, groups, kind):
    """At most one row of K sums per CTA for each parameter, at most 152 x 8 CTAs: the size is bounded
    whatever M, and it is a whole number of rows of three (or two) sums."""
    n = L.nvfp4_residual_norm_backward_workspace_bytes(M, K, groups, kind)
    row = 4 * K
    assert 2 * row <= n <= 3 * (152 * 8 * row + 256)


def test_valid_calls_without_a_gpu_fail_cleanly(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    buf = ctypes.create_string_buffer(1 << 16)
    p = (ctypes.addressof(buf) + 255) & ~255
    o = p + (1 << 15)
    calls = [("nvfp4_fp8_quantize_act", (p, BF, 4, 256, 256, p, p, 4, None)),
             ("nvfp4_fp8_gemm", (p, p, 4, 4, 256, 8, p, p, BF, o, None)),
             ("nvfp4_gated_linear", (p, BF, 4, 64, 64, 16, p, p, 0, o, None, None)),
             ("nvfp4_residual_norm", (p, BF, p, BF, 4, 64, 64, 64, None, None, 0, 0, 1.0, None, 1e-6, o, None, None, None))]
    for name, args in calls:
        assert getattr(L, name)(*args) in (_lib.ERR_CUDA, _lib.ERR_UNSUPPORTED_DEVICE)


def test_torch_layer_refuses_cpu_tensors():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(16, 64, dtype=torch.bfloat16)
    for f in [lambda: ops.fp8_quantize_act(x), lambda: ops.gated_linear(x, w, w), lambda: ops.residual_norm(x, x)]:
        with pytest.raises(ValueError, match="CUDA"):
            f()


def test_stats_in_place_are_refused(L):
    """The backward reads r: a forward that keeps statistics for it may not overwrite r with r_out."""
    a = dict(f=P, dtype=BF, r=4 * P, rd=BF, M=6, K=64, ldf=64, ldr=64, ga=None, gate=None, kind=0, groups=0, scale=1.0, gb=None, eps=1e-6,
             ro=4 * P, y=None, stats=8 * P, stream=None)
    refuses(L, "nvfp4_residual_norm", changed(a), 1)
    assert b"backward" in L.nvfp4_last_error_string()


# every operand of a call in a range of its own: (name, bytes); written ones are moved into each of the others below
CALLS = {
    "nvfp4_fp8_quantize_weight": (dict(w=0, dtype=BF, N=200, K=256, ldw=272, q=0, w_s=0, stream=None),
                                  dict(w=(199 * 272 + 256) * 2, q=200 * 256, w_s=16), ["q", "w_s"]),
    "nvfp4_fp8_gemm": (dict(xq=0, xs=0, lds=8, M=5, K=256, N=200, w=0, w_s=0, dtype=BF, y=0, stream=None),
                       dict(xq=5 * 256, xs=(8 + 5) * 4, w=200 * 256, w_s=16, y=5 * 200 * 2), ["y"]),
    "nvfp4_fp8_linear": (dict(x=0, dtype=HF, M=70, K=256, ldx=264, N=200, w=0, w_s=0, y=0, ws=0, bytes=1 << 15, stream=None),
                         dict(x=(69 * 264 + 256) * 2, w=200 * 256, w_s=16, y=70 * 200 * 2, ws=70 * 256 + 2 * 72 * 4), ["y", "ws"]),
    "nvfp4_gated_linear": (dict(x=0, dtype=BF, T=5, H=64, ldx=72, I=16, wg=0, wu=0, act=0, h=0, gu=0, stream=None),
                           dict(x=(4 * 72 + 64) * 2, wg=16 * 64 * 2, wu=16 * 64 * 2, h=5 * 16 * 2, gu=5 * 32 * 4), ["h", "gu"]),
    "nvfp4_gated_linear_backward": (
        dict(dh=0, lddh=24, x=0, ldx=72, dtype=BF, T=5, H=64, I=16, wg=0, wu=0, act=0, gu=0, dx=0, dwg=0, dwu=0, ws=0, bytes=512, stream=None),
        dict(dh=(4 * 24 + 16) * 2, x=(4 * 72 + 64) * 2, wg=16 * 64 * 2, wu=16 * 64 * 2, gu=5 * 32 * 4, dx=5 * 64 * 2, dwg=16 * 64 * 2,
             dwu=16 * 64 * 2, ws=512), ["dx", "dwg", "dwu", "ws"]),
    "nvfp4_residual_norm": (
        dict(f=0, dtype=BF, r=0, rd=F32, M=6, K=64, ldf=72, ldr=80, ga=0, gate=0, kind=1, groups=3, scale=1.0, gb=0, eps=1e-6, ro=0, y=0,
             stats=0, stream=None),
        dict(f=(5 * 72 + 64) * 2, r=(5 * 80 + 64) * 4, ga=128, gate=3 * 128, gb=128, ro=6 * 64 * 4, y=6 * 64 * 2, stats=6 * 8),
        ["ro", "y", "stats"]),
    "nvfp4_residual_norm_backward": (
        dict(dro=0, lddr=72, dy=0, lddy=80, f=0, dtype=BF, r=0, rd=BF, M=6, K=64, ldf=64, ldr=64, stats=0, ga=0, gate=0, kind=2, groups=1,
             scale=1.0, gb=0, df=0, dr=0, dga=0, dgate=0, dgb=0, ws=0, bytes=1 << 15, stream=None),
        dict(dro=(5 * 72 + 64) * 2, dy=(5 * 80 + 64) * 2, f=6 * 128, r=6 * 128, stats=6 * 8, ga=128, gate=6 * 2, gb=128, df=6 * 128,
             dr=6 * 128, dga=256, dgate=6 * 4, dgb=256, ws=1024), ["df", "dr", "dga", "dgate", "dgb", "ws"]),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_nothing_written_overlaps_another_operand(L, name):
    """Each output and the workspace at the first and in the last 256 bytes of every other operand, and with its own last
    byte on the other's first; apart from each other the call gets past its checks."""
    base, sizes, written = CALLS[name]
    at = {o: P + (i << 20) for i, o in enumerate(sizes)}
    base = {**base, **at}
    if not torch.cuda.is_available():  # the pointers are not real: the call ends at the device
        assert getattr(L, name)(*changed(base)) in (_lib.ERR_CUDA, _lib.ERR_UNSUPPORTED_DEVICE)
    for w in written:
        for o, n in sizes.items():
            if o == w:
                continue
            for p in (at[o], at[o] + (n - 1) // 256 * 256, at[o] - (sizes[w] - 1) // 256 * 256):
                if (w, o) == ("ro", "r") and p == at["r"]:
                    continue  # in place: allowed or refused by rules of its own (stride, statistics)
                refuses(L, name, changed(base, **{w: p}), 1)
                assert b"overlap" in L.nvfp4_last_error_string(), (w, o)
    if name == "nvfp4_residual_norm":  # r_out may be r itself (same stride), without statistics
        same = changed(base, ro=at["r"], ldr=64, stats=None)
        if not torch.cuda.is_available():
            assert getattr(L, name)(*same) in (_lib.ERR_CUDA, _lib.ERR_UNSUPPORTED_DEVICE)


def test_a_gate_of_no_rows_has_no_address(L):
    if torch.cuda.is_available():
        pytest.skip("the pointers are not real")
    a = dict(f=None, dtype=BF, r=None, rd=BF, M=0, K=64, ldf=64, ldr=64, ga=None, gate=None, kind=2, groups=0, scale=1.0, gb=None, eps=1e-6,
             ro=None, y=None, stats=None, stream=None)
    assert L.nvfp4_residual_norm(*changed(a)) in (_lib.ERR_CUDA, _lib.ERR_UNSUPPORTED_DEVICE)
    refuses(L, "nvfp4_residual_norm", changed(a, M=1, f=P, r=2 * P, ro=3 * P), 1)
