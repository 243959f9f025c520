"""Torch-facing wrappers of the C ABI (argument marshalling only).

Every function takes and returns CUDA tensors; outputs are allocated with
torch (device memory plumbing) and every step of the computation runs in the
library's kernels.  Tensors on any other device are rejected: there is no CPU
path.
"""

from __future__ import annotations

from dataclasses import dataclass
from typing import Optional, Tuple

import torch

from . import _lib
from ._lib import call, lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream: Optional[torch.cuda.Stream] = None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _cuda(*tensors: Optional[torch.Tensor]) -> None:
    for t in tensors:
        if t is not None and not t.is_cuda:
            raise ValueError("nvfp4 ops take CUDA tensors only (no CPU fallback)")
        if t is not None and not t.is_contiguous():
            raise ValueError("nvfp4 ops take contiguous tensors")


def _u8(*shape: int, device) -> torch.Tensor:
    return torch.empty(*shape, dtype=torch.uint8, device=device)


def sf_bytes(rows: int, K: int) -> int:
    return int(lib().nvfp4_sf_bytes(rows, K))


# --------------------------------------------------------------------------- (a) quantize

def quantize_act(x: torch.Tensor, gs: Optional[torch.Tensor] = None, sf_layout: str = "swizzled",
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """x (M, K) bf16 -> (q (M, K/2) uint8, sf uint8, gs (1,) fp32).

    ``gs=None`` computes the dynamic global scale amax/2688 on the device;
    a given ``gs`` (device fp32 scalar tensor) is used as a static scale.
    """
    _cuda(x, gs)
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise ValueError("x must be a 2-D bf16 tensor")
    M, K = x.shape
    layout = _lib.SF_SWIZZLED if sf_layout == "swizzled" else _lib.SF_LINEAR
    q = _u8(M, K // 2, device=x.device)
    sf = _u8(sf_bytes(M, K) if layout == _lib.SF_SWIZZLED else M * (K // 16), device=x.device)
    dyn = gs is None
    gs_t = torch.empty(1, dtype=torch.float32, device=x.device) if dyn else gs
    ws_n = int(lib().nvfp4_quantize_workspace_bytes(M, K))
    ws = _u8(ws_n, device=x.device) if dyn else None
    call("nvfp4_quantize_act", x.data_ptr(), M, K, K, _lib.GS_DYNAMIC if dyn else _lib.GS_STATIC, gs_t.data_ptr(),
         q.data_ptr(), sf.data_ptr(), layout, _ptr(ws), ws_n if dyn else 0, _stream(stream))
    return q, sf, gs_t


def rmsnorm(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6, stream=None) -> torch.Tensor:
    """x (M, K) bf16 -> x / rms(x) * gamma, bf16 (the unfused normalisation)."""
    _cuda(x, gamma)
    M, K = x.shape
    y = torch.empty_like(x)
    call("nvfp4_rmsnorm", x.data_ptr(), M, K, K, gamma.data_ptr(), eps, y.data_ptr(), _stream(stream))
    return y


def rmsnorm_quantize(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6, gs: Optional[torch.Tensor] = None,
                     sf_layout: str = "swizzled", want_normed: bool = False, stream=None):
    """Fused RMSNorm -> NVFP4: returns (q, sf, gs, x_normed or None)."""
    _cuda(x, gamma, gs)
    M, K = x.shape
    layout = _lib.SF_SWIZZLED if sf_layout == "swizzled" else _lib.SF_LINEAR
    q = _u8(M, K // 2, device=x.device)
    sf = _u8(sf_bytes(M, K) if layout == _lib.SF_SWIZZLED else M * (K // 16), device=x.device)
    dyn = gs is None
    gs_t = torch.empty(1, dtype=torch.float32, device=x.device) if dyn else gs
    xn = torch.empty_like(x) if want_normed else None
    ws_n = int(lib().nvfp4_rmsnorm_quantize_workspace_bytes(M, K))
    ws = _u8(ws_n, device=x.device)
    call("nvfp4_rmsnorm_quantize", x.data_ptr(), M, K, K, gamma.data_ptr(), eps,
         _lib.GS_DYNAMIC if dyn else _lib.GS_STATIC, gs_t.data_ptr(), q.data_ptr(), sf.data_ptr(), layout,
         _ptr(xn), ws.data_ptr(), ws_n, _stream(stream))
    return q, sf, gs_t, xn


def prepare_weights(w: torch.Tensor, sf: torch.Tensor, N: int, K: int, interleave_w13: bool = False,
                    stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Checkpoint codes (G, N, K/2) + row-major scales (G, N, K/16) -> prepared (tile-major) codes
    + swizzled scales."""
    _cuda(w, sf)
    G = w.numel() // (N * K // 2)
    w_out = _u8(int(lib().nvfp4_prepared_weight_bytes(G, N, K)), device=w.device)
    sf_out = _u8(G * sf_bytes(N, K), device=w.device)
    call("nvfp4_prepare_weights", w.data_ptr(), sf.data_ptr(), G, N, K,
         _lib.PREP_W13_INTERLEAVE if interleave_w13 else _lib.PREP_PLAIN, w_out.data_ptr(), sf_out.data_ptr(),
         _stream(stream))
    return w_out, sf_out


# --------------------------------------------------------------------------- (e) dense linear

def linear(x: torch.Tensor, w: torch.Tensor, w_sf: torch.Tensor, ws2: torch.Tensor, N: int,
           gs: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
           stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """y (M, N) bf16 = (gs * ws2) * deq(quantize(x)) @ deq(W)^T; returns (y, gs)."""
    _cuda(x, w, w_sf, ws2, gs, workspace)
    M, K = x.shape
    y = torch.empty(M, N, dtype=torch.bfloat16, device=x.device)
    dyn = gs is None
    gs_t = torch.empty(1, dtype=torch.float32, device=x.device) if dyn else gs
    ws_n = int(lib().nvfp4_linear_workspace_bytes(M, K))
    ws = workspace if workspace is not None else _u8(ws_n, device=x.device)
    call("nvfp4_linear", x.data_ptr(), M, K, N, w.data_ptr(), w_sf.data_ptr(), ws2.data_ptr(),
         _lib.GS_DYNAMIC if dyn else _lib.GS_STATIC, gs_t.data_ptr(), y.data_ptr(), ws.data_ptr(), ws.numel(),
         _stream(stream))
    return y, gs_t


def grouped_linear(x: torch.Tensor, w: torch.Tensor, w_sf: torch.Tensor, ws2: torch.Tensor, G: int, N: int,
                   gs: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """x (M, G*K) bf16, W (G, N, K/2) prepared -> y (M, G*N) bf16; group g uses x's K columns g."""
    _cuda(x, w, w_sf, ws2, gs, workspace)
    M, GK = x.shape
    K = GK // G
    y = torch.empty(M, G * N, dtype=torch.bfloat16, device=x.device)
    dyn = gs is None
    gs_t = torch.empty(1, dtype=torch.float32, device=x.device) if dyn else gs
    ws_n = int(lib().nvfp4_grouped_linear_workspace_bytes(M, G, K))
    ws = workspace if workspace is not None else _u8(ws_n, device=x.device)
    call("nvfp4_grouped_linear", x.data_ptr(), M, G, K, N, w.data_ptr(), w_sf.data_ptr(), ws2.data_ptr(),
         _lib.GS_DYNAMIC if dyn else _lib.GS_STATIC, gs_t.data_ptr(), y.data_ptr(), ws.data_ptr(), ws.numel(),
         _stream(stream))
    return y, gs_t


def gemm(xq: torch.Tensor, xsf: torch.Tensor, gs: torch.Tensor, K: int, w: torch.Tensor, w_sf: torch.Tensor,
         ws2: torch.Tensor, N: int, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """GEMM alone on quantised activations xq (M, K/2) + swizzled xsf."""
    _cuda(xq, xsf, gs, w, w_sf, ws2, out)
    M = xq.shape[0]
    y = out if out is not None else torch.empty(M, N, dtype=torch.bfloat16, device=xq.device)
    call("nvfp4_gemm", xq.data_ptr(), xsf.data_ptr(), gs.data_ptr(), M, K, N, w.data_ptr(), w_sf.data_ptr(),
         ws2.data_ptr(), y.data_ptr(), _stream(stream))
    return y


# --------------------------------------------------------------------------- router gate

def router_prepare(w: torch.Tensor, w_sf_linear: torch.Tensor, ws2: torch.Tensor, E: int, H: int,
                   stream=None) -> torch.Tensor:
    """NVFP4 gate weight (E, H/2) + row-major scales -> bf16 weight after the FP8-E4M3 round trip."""
    _cuda(w, w_sf_linear, ws2)
    wg = torch.empty(E, H, dtype=torch.bfloat16, device=w.device)
    n = int(lib().nvfp4_router_prepare_workspace_bytes(E, H))
    ws = _u8(n, device=w.device)
    call("nvfp4_router_prepare", w.data_ptr(), w_sf_linear.data_ptr(), ws2.data_ptr(), E, H, wg.data_ptr(),
         ws.data_ptr(), n, _stream(stream))
    return wg


def router(x: torch.Tensor, wg: torch.Tensor, topk: int, want_logits: bool = False, stream=None):
    """Dense router: (ids (T, topk) int32, weights (T, topk) fp32, logits (T, E) fp32 or None)."""
    _cuda(x, wg)
    T, H = x.shape
    E = wg.shape[0]
    ids = torch.empty(T, topk, dtype=torch.int32, device=x.device)
    w = torch.empty(T, topk, dtype=torch.float32, device=x.device)
    logits = torch.empty(T, E, dtype=torch.float32, device=x.device) if want_logits else None
    n = int(lib().nvfp4_router_workspace_bytes(T, E))
    ws = _u8(max(n, 256), device=x.device)
    call("nvfp4_router", x.data_ptr(), T, H, wg.data_ptr(), E, topk, ids.data_ptr(), w.data_ptr(), _ptr(logits),
         ws.data_ptr(), ws.numel(), _stream(stream))
    return ids, w, logits


# --------------------------------------------------------------------------- (b) routing

def moe_route(ids: torch.Tensor, E: int, stream=None):
    """ids (T, k) int32 -> counts (E,), offsets (E+1,), sorted_idx (T*k,), inv_idx (T*k,)."""
    _cuda(ids)
    T, k = ids.shape
    dev = ids.device
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    sorted_idx = torch.empty(max(T * k, 1), dtype=torch.int32, device=dev)
    inv_idx = torch.empty(max(T * k, 1), dtype=torch.int32, device=dev)
    call("nvfp4_moe_route", ids.data_ptr(), T, k, E, counts.data_ptr(), offsets.data_ptr(), sorted_idx.data_ptr(),
         inv_idx.data_ptr(), _stream(stream))
    return counts, offsets, sorted_idx[: T * k], inv_idx[: T * k]


# --------------------------------------------------------------------------- MoE layer

@dataclass
class MoEWeights:
    """Prepared expert weights (see nvfp4_prepare_weights) and their ws2 scalars."""
    E: int
    H: int
    I: int
    w13: torch.Tensor       # (E, 2I, H/2) interleaved
    w13_sf: torch.Tensor
    w13_ws2: torch.Tensor   # (E,) fp32
    w2: torch.Tensor        # (E, H, I/2)
    w2_sf: torch.Tensor
    w2_ws2: torch.Tensor    # (E,)
    sh_w13: Optional[torch.Tensor] = None
    sh_w13_sf: Optional[torch.Tensor] = None
    sh_w2: Optional[torch.Tensor] = None
    sh_w2_sf: Optional[torch.Tensor] = None
    sh_ws2: Optional[torch.Tensor] = None  # (2,) = (w13 ws2, w2 ws2)

    @property
    def has_shared(self) -> bool:
        return self.sh_w13 is not None


def moe_workspace_layout(T: int, H: int, I: int, E: int, topk: int, has_shared: bool) -> _lib.MoeWsLayout:
    L = _lib.MoeWsLayout()
    call("nvfp4_moe_workspace_layout", T, H, I, E, topk, int(has_shared), _lib.ctypes.byref(L))
    return L


def moe_workspace(T: int, H: int, I: int, E: int, topk: int, has_shared: bool, device) -> torch.Tensor:
    n = int(lib().nvfp4_moe_workspace_bytes(T, H, I, E, topk, int(has_shared)))
    if n == 0:
        raise ValueError("unsupported MoE shape")
    return _u8(n, device=device)


def _wp(W: MoEWeights):
    return (W.w13.data_ptr(), W.w13_sf.data_ptr(), W.w13_ws2.data_ptr(), W.w2.data_ptr(), W.w2_sf.data_ptr(),
            W.w2_ws2.data_ptr(), _ptr(W.sh_w13), _ptr(W.sh_w13_sf), _ptr(W.sh_w2), _ptr(W.sh_w2_sf),
            _ptr(W.sh_ws2))


def moe_forward(x: torch.Tensor, ids: torch.Tensor, topk_w: torch.Tensor, W: MoEWeights, a2_gs: torch.Tensor,
                a1_gs: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Routed MoE + shared expert.  Returns (y (T, H) bf16, a1_gs)."""
    _cuda(x, ids, topk_w, a2_gs, a1_gs, workspace, out)
    T, H = x.shape
    k = ids.shape[1]
    dyn = a1_gs is None
    gs_t = torch.empty(1, dtype=torch.float32, device=x.device) if dyn else a1_gs
    ws = workspace if workspace is not None else moe_workspace(T, H, W.I, W.E, k, W.has_shared, x.device)
    y = out if out is not None else torch.empty(T, H, dtype=torch.bfloat16, device=x.device)
    call("nvfp4_moe_forward", x.data_ptr(), T, H, W.I, W.E, k, ids.data_ptr(), topk_w.data_ptr(), *_wp(W),
         _lib.GS_DYNAMIC if dyn else _lib.GS_STATIC, gs_t.data_ptr(), a2_gs.data_ptr(), y.data_ptr(),
         ws.data_ptr(), ws.numel(), _stream(stream))
    return y, gs_t


def moe_dispatch(x, ids, W: MoEWeights, a1_gs: torch.Tensor, dynamic: bool, workspace: torch.Tensor, stream=None):
    T, H = x.shape
    call("nvfp4_moe_dispatch", x.data_ptr(), T, H, W.I, W.E, ids.shape[1], ids.data_ptr(), int(W.has_shared),
         _lib.GS_DYNAMIC if dynamic else _lib.GS_STATIC, a1_gs.data_ptr(), workspace.data_ptr(), workspace.numel(),
         _stream(stream))


def moe_w13(T: int, topk: int, W: MoEWeights, a1_gs, a2_gs, workspace, h_debug=None, stream=None):
    call("nvfp4_moe_w13", T, W.H, W.I, W.E, topk, W.w13.data_ptr(), W.w13_sf.data_ptr(), W.w13_ws2.data_ptr(),
         _ptr(W.sh_w13), _ptr(W.sh_w13_sf), _ptr(W.sh_ws2), a1_gs.data_ptr(), a2_gs.data_ptr(), _ptr(h_debug),
         workspace.data_ptr(), workspace.numel(), _stream(stream))


def moe_w2(T: int, topk: int, topk_w, W: MoEWeights, a2_gs, workspace, stream=None):
    call("nvfp4_moe_w2", T, W.H, W.I, W.E, topk, topk_w.data_ptr(), W.w2.data_ptr(), W.w2_sf.data_ptr(),
         W.w2_ws2.data_ptr(), _ptr(W.sh_w2), _ptr(W.sh_w2_sf), _ptr(W.sh_ws2), a2_gs.data_ptr(),
         workspace.data_ptr(), workspace.numel(), _stream(stream))


def moe_finalize(T: int, topk: int, W: MoEWeights, y, workspace, stream=None):
    call("nvfp4_moe_finalize", T, W.H, W.I, W.E, topk, int(W.has_shared), y.data_ptr(), workspace.data_ptr(),
         workspace.numel(), _stream(stream))


# --------------------------------------------------------------------------- dense feed-forward operators
#
# The operators around the experts: bf16 or fp16 tensors, rows with any stride that is a multiple of
# 8 elements where a call says "strided rows", everything else contiguous.  They keep no autograd
# graph: a backward pass is its own call.  With ``stream`` given, outputs and scratch are allocated
# for that stream and the inputs are marked as used on it.

_DT = {torch.bfloat16: _lib.DT_BF16, torch.float16: _lib.DT_FP16}
_ACT = {"silu": _lib.ACT_SILU, "gelu": _lib.ACT_GELU, "gelu_tanh": _lib.ACT_GELU_TANH}
_CODES = (torch.float8_e4m3fn, torch.uint8)


class _Place:
    """The device of a call's tensors (all the same) as the current one, and its stream."""

    def __init__(self, stream, *tensors: Optional[torch.Tensor]):
        first = tensors[0]
        for t in tensors:
            if t is None:
                continue
            if not t.is_cuda:
                raise ValueError("nvfp4 ops take CUDA tensors only (no CPU fallback)")
            if t.device != first.device:
                raise ValueError("tensors on different devices")
        self.device = first.device
        self._guards = []
        if first.get_device() != torch.cuda.current_device():
            self._guards.append(torch.cuda.device(first.device))
        if stream is not None:
            if stream.device != first.device:
                raise ValueError("stream of another device")
            self._guards.append(torch.cuda.stream(stream))
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)

    def __enter__(self):
        for g in self._guards:
            g.__enter__()
        return torch.cuda.current_stream().cuda_stream

    def __exit__(self, *exc):
        for g in reversed(self._guards):
            g.__exit__(*exc)


def _kind(x: torch.Tensor, what: str) -> int:
    d = _DT.get(x.dtype)
    if d is None:
        raise ValueError(f"{what} must be bf16 or fp16, got {x.dtype}")
    return d


def _ld(t: torch.Tensor, what: str, rows: Optional[int] = None, cols: Optional[int] = None, dtype=None) -> int:
    """Row stride of a 2-D tensor of strided rows (a single row's stride does not matter)."""
    if t.dim() != 2 or (rows is not None and t.shape[0] != rows) or (cols is not None and t.shape[1] != cols):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected ({rows if rows is not None else 'rows'}, "
                         f"{cols if cols is not None else 'columns'})")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{what}: the elements of a row must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _whole(t: torch.Tensor, what: str, shape, dtypes) -> int:
    """Data pointer of a contiguous tensor of the given shape and type."""
    if tuple(t.shape) != tuple(shape) or t.dtype not in dtypes:
        raise ValueError(f"{what} has shape {tuple(t.shape)} and type {t.dtype}, expected {tuple(shape)} {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def fp8_quantize_act(x: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """x (M, K) strided rows -> (q (M, K) float8_e4m3fn, s (ceil(K / 128), M) fp32).

    One scale per 128 consecutive K elements of a row, s = max|x| / 448, q = e4m3(x / s).  s is a view
    of rows padded to a multiple of four, as ``fp8_gemm`` wants them.  K % 16 == 0.
    """
    with _Place(stream, x) as st:
        ld = _ld(x, "x")
        M, K = x.shape
        q = torch.empty(M, K, dtype=torch.float8_e4m3fn, device=x.device)
        lds = (M + 3) // 4 * 4
        s = torch.empty((K + 127) // 128, lds, dtype=torch.float32, device=x.device)
        call("nvfp4_fp8_quantize_act", x.data_ptr(), _kind(x, "x"), M, K, ld, q.data_ptr(), s.data_ptr(), lds, st)
        return q, s[:, :M]


def fp8_quantize_weight(w: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """w (N, K) strided rows -> (q (N, K) float8_e4m3fn, s (ceil(N / 128), ceil(K / 128)) fp32): one
    scale per 128 x 128 block, the layout checkpoints store.  Once, at load time.  K % 16 == 0."""
    with _Place(stream, w) as st:
        ld = _ld(w, "w")
        N, K = w.shape
        q = torch.empty(N, K, dtype=torch.float8_e4m3fn, device=w.device)
        s = torch.empty((N + 127) // 128, (K + 127) // 128, dtype=torch.float32, device=w.device)
        call("nvfp4_fp8_quantize_weight", w.data_ptr(), _kind(w, "w"), N, K, ld, q.data_ptr(), s.data_ptr(), st)
        return q, s


def _fp8_weight(w: torch.Tensor, w_s: torch.Tensor, K: int) -> Tuple[int, int, int]:
    if w.dim() != 2:
        raise ValueError("w must be 2-D")
    N = w.shape[0]
    return (N, _whole(w, "w", (N, K), _CODES),
            _whole(w_s, "w_s", ((N + 127) // 128, (K + 127) // 128), (torch.float32,)))


def fp8_gemm(xq: torch.Tensor, xs: torch.Tensor, w: torch.Tensor, w_s: torch.Tensor, dtype=torch.bfloat16,
             out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y (M, N) = deq(xq) deq(w)^T of quantised activations (``fp8_quantize_act``) and weights, in
    bf16 or fp16; the scales apply to fp32 sums of one 128-wide K block each."""
    with _Place(stream, xq, xs, w, w_s, out) as st:
        if xq.dim() != 2 or xs.dim() != 2:
            raise ValueError("xq and xs must be 2-D")
        M, K = xq.shape
        N, wp, wsp = _fp8_weight(w, w_s, K)
        KB = (K + 127) // 128
        lds = xs.stride(0) if KB > 1 else max(xs.stride(0), (M + 3) // 4 * 4)
        room = xs.untyped_storage().nbytes() // 4 - xs.storage_offset()
        if xs.dtype != torch.float32 or tuple(xs.shape) != (KB, M) or (M > 1 and xs.stride(1) != 1):
            raise ValueError(f"xs must be fp32 ({KB}, {M}) with contiguous rows")
        if M and room < (KB - 1) * lds + (M + 3) // 4 * 4:
            raise ValueError("the rows of xs must be padded to a multiple of four scales")
        if dtype not in _DT:
            raise ValueError(f"output type {dtype}")
        y = out if out is not None else torch.empty(M, N, dtype=dtype, device=xq.device)
        call("nvfp4_fp8_gemm", _whole(xq, "xq", (M, K), _CODES), xs.data_ptr(), lds, M, K, N, wp, wsp, _DT[dtype],
             _whole(y, "out", (M, N), (dtype,)), st)
        return y


def fp8_linear(x: torch.Tensor, w: torch.Tensor, w_s: torch.Tensor, out: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y (M, N) = deq(quantize(x)) deq(w)^T in x's type: x (M, K) strided rows, w (N, K) e4m3 codes
    with w_s (ceil(N / 128), ceil(K / 128)) fp32 scales as checkpoints store them."""
    with _Place(stream, x, w, w_s, out, workspace) as st:
        ld = _ld(x, "x")
        M, K = x.shape
        N, wp, wsp = _fp8_weight(w, w_s, K)
        y = out if out is not None else torch.empty(M, N, dtype=x.dtype, device=x.device)
        n = int(lib().nvfp4_fp8_linear_workspace_bytes(M, K))
        ws = workspace if workspace is not None else _u8(n, device=x.device)
        call("nvfp4_fp8_linear", x.data_ptr(), _kind(x, "x"), M, K, ld, N, wp, wsp,
             _whole(y, "out", (M, N), (x.dtype,)), _whole(ws, "workspace", (ws.numel(),), (torch.uint8,)), ws.numel(),
             st)
        return y


def _gated_args(x, w_gate, w_up, activation):
    if activation not in _ACT:
        raise ValueError(f"activation {activation!r}, expected one of {sorted(_ACT)}")
    ld = _ld(x, "x")
    if w_gate.dim() != 2:
        raise ValueError("w_gate must be 2-D")
    T, H = x.shape
    I = w_gate.shape[0]
    return (T, H, I, ld, _kind(x, "x"), _whole(w_gate, "w_gate", (I, H), (x.dtype,)),
            _whole(w_up, "w_up", (I, H), (x.dtype,)), _ACT[activation])


def gated_linear(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, activation: str = "silu",
                 save: bool = False, out: Optional[torch.Tensor] = None, stream=None):
    """h (T, I) = act(x w_gate^T) * (x w_up^T): x (T, H) strided rows, weights (I, H), one type.

    ``activation``: "silu", "gelu" (erf) or "gelu_tanh".  With ``save`` returns (h, gu), gu (T, 2I) the
    fp32 pre-activations [g | u] that ``gated_linear_backward`` takes.  H % 8 == 0, I % 8 == 0.
    """
    with _Place(stream, x, w_gate, w_up, out) as st:
        T, H, I, ld, kind, gp, up, act = _gated_args(x, w_gate, w_up, activation)
        h = out if out is not None else torch.empty(T, I, dtype=x.dtype, device=x.device)
        gu = torch.empty(T, 2 * I, dtype=torch.float32, device=x.device) if save else None
        call("nvfp4_gated_linear", x.data_ptr(), kind, T, H, ld, I, gp, up, act, _whole(h, "out", (T, I), (x.dtype,)),
             _ptr(gu), st)
        return (h, gu) if save else h


def gated_linear_backward(dh: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
                          gu: torch.Tensor, activation: str = "silu", need_dx: bool = True, need_dw: bool = True,
                          workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients (dx (T, H), dw_gate (I, H), dw_up (I, H)) of ``gated_linear`` from dh (T, I) strided
    rows and the saved gu; those not asked for are None."""
    with _Place(stream, x, dh, w_gate, w_up, gu, workspace) as st:
        T, H, I, ld, kind, gp, up, act = _gated_args(x, w_gate, w_up, activation)
        lddh = _ld(dh, "dh", T, I, x.dtype)
        gup = _whole(gu, "gu", (T, 2 * I), (torch.float32,))
        dx = torch.empty(T, H, dtype=x.dtype, device=x.device) if need_dx else None
        dwg = torch.empty(I, H, dtype=x.dtype, device=x.device) if need_dw else None
        dwu = torch.empty(I, H, dtype=x.dtype, device=x.device) if need_dw else None
        n = int(lib().nvfp4_gated_linear_backward_workspace_bytes(T, I))
        ws = workspace if workspace is not None else _u8(n, device=x.device)
        call("nvfp4_gated_linear_backward", dh.data_ptr(), lddh, x.data_ptr(), ld, kind, T, H, I, gp, up, act, gup,
             _ptr(dx), _ptr(dwg), _ptr(dwu), _whole(ws, "workspace", (ws.numel(),), (torch.uint8,)), ws.numel(), st)
        return dx, dwg, dwu


def _norm_args(f, r, gamma_after, gate, gamma_before):
    ldf, kind = _ld(f, "f"), _kind(f, "f")
    M, K = f.shape
    if r.dtype != f.dtype and r.dtype != torch.float32:
        raise ValueError(f"r must be {f.dtype} or fp32, got {r.dtype}")
    ldr = _ld(r, "r", M, K)
    rkind = _lib.DT_FP32 if r.dtype == torch.float32 else kind
    ga = None if gamma_after is None else _whole(gamma_after, "gamma_after", (K,), (f.dtype,))
    gb = None if gamma_before is None else _whole(gamma_before, "gamma_before", (K,), (f.dtype,))
    if gate is None:
        return M, K, ldf, ldr, kind, rkind, ga, None, _lib.GATE_NONE, 0, gb
    if gate.dim() == 2 and tuple(gate.shape) == (M, 1):
        return M, K, ldf, ldr, kind, rkind, ga, _whole(gate, "gate", (M, 1), (f.dtype,)), _lib.GATE_ROW, 0, gb
    groups = 1 if gate.dim() == 1 else gate.shape[0]
    gp = _whole(gate, "gate", (K,) if gate.dim() == 1 else (groups, K), (f.dtype,))
    if groups == 0 or M % groups:
        raise ValueError(f"{M} rows do not split into {groups} groups")
    return M, K, ldf, ldr, kind, rkind, ga, gp, _lib.GATE_CHANNEL, groups, gb


def residual_norm(f: torch.Tensor, r: torch.Tensor, gamma_after: Optional[torch.Tensor] = None,
                  gate: Optional[torch.Tensor] = None, scale: float = 1.0,
                  gamma_before: Optional[torch.Tensor] = None, eps: float = 1e-6, save: bool = False,
                  out: Optional[torch.Tensor] = None, stream=None):
    """The boundary between two blocks: returns (r_out, y), with ``save`` (r_out, y, stats).

    n = rmsnorm(f; gamma_after) (f without gamma_after), r_out = r + scale * gate * n, y =
    rmsnorm(r_out; gamma_before) from the unrounded sum (None without gamma_before).  f (M, K) and r
    (M, K; f's type or fp32) strided rows; gate (K,), (groups, K) for M / groups consecutive rows each,
    or (M, 1).  ``out`` receives r_out and may be r.  K % 8 == 0, K <= 16384.
    """
    with _Place(stream, f, r, gamma_after, gate, gamma_before, out) as st:
        M, K, ldf, ldr, kind, rkind, ga, gp, gkind, groups, gb = _norm_args(f, r, gamma_after, gate, gamma_before)
        r_out = out if out is not None else torch.empty(M, K, dtype=r.dtype, device=f.device)
        y = torch.empty(M, K, dtype=f.dtype, device=f.device) if gb is not None else None
        stats = torch.empty(M, 2, dtype=torch.float32, device=f.device) if save else None
        call("nvfp4_residual_norm", f.data_ptr(), kind, r.data_ptr(), rkind, M, K, ldf, ldr, ga, gp, gkind, groups, scale,
             gb, eps, _whole(r_out, "out", (M, K), (r.dtype,)), _ptr(y), _ptr(stats), st)
        return (r_out, y, stats) if save else (r_out, y)


def residual_norm_backward(dr_out: Optional[torch.Tensor], dy: Optional[torch.Tensor], f: torch.Tensor,
                           r: torch.Tensor, stats: torch.Tensor, gamma_after: Optional[torch.Tensor] = None,
                           gate: Optional[torch.Tensor] = None, scale: float = 1.0,
                           gamma_before: Optional[torch.Tensor] = None, eps: float = 1e-6,
                           workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients (df, dr, dgamma_after, dgate, dgamma_before) of ``residual_norm``; the parameters' are
    fp32 in their own shapes, None where the parameter is absent.

    dr_out (r's type) and dy (f's type) are the gradients of r_out and y, strided rows; either may be
    None (zero).  The other arguments are the forward's (eps is already in ``stats``).
    """
    with _Place(stream, f, r, dr_out, dy, stats, gamma_after, gate, gamma_before, workspace) as st:
        M, K, ldf, ldr, kind, rkind, ga, gp, gkind, groups, gb = _norm_args(f, r, gamma_after, gate, gamma_before)
        if dy is not None and gb is None:
            raise ValueError("dy without gamma_before")
        lddr = K if dr_out is None else _ld(dr_out, "dr_out", M, K, r.dtype)
        lddy = K if dy is None else _ld(dy, "dy", M, K, f.dtype)
        sp = _whole(stats, "stats", (M, 2), (torch.float32,))
        df = torch.empty(M, K, dtype=f.dtype, device=f.device)
        dr = torch.empty(M, K, dtype=r.dtype, device=f.device)

        def grad(p):
            return None if p is None else torch.empty(p.shape, dtype=torch.float32, device=f.device)

        dga, dgate, dgb = grad(gamma_after), grad(gate), grad(gamma_before)
        n = int(lib().nvfp4_residual_norm_backward_workspace_bytes(M, K, max(groups, 1), rkind))
        ws = workspace if workspace is not None else _u8(n, device=f.device)
        call("nvfp4_residual_norm_backward", _ptr(dr_out), lddr, _ptr(dy), lddy, f.data_ptr(), kind, r.data_ptr(), rkind,
             M, K, ldf, ldr, sp, ga, gp, gkind, groups, scale, gb, df.data_ptr(), dr.data_ptr(), _ptr(dga), _ptr(dgate),
             _ptr(dgb), _whole(ws, "workspace", (ws.numel(),), (torch.uint8,)), ws.numel(), st)
        return df, dr, dga, dgate, dgb


# --------------------------------------------------------------------------- diagnostics

def device_error(stream=None) -> Tuple[int, int]:
    """(status, flags) of the device fault word; synchronises the stream and clears the flags."""
    flags = _lib.ctypes.c_int32(0)
    st = lib().nvfp4_get_device_error(_stream(stream), _lib.ctypes.byref(flags))
    return int(st), int(flags.value)


def debug_wait_timeout(timeout_us: int, stream=None) -> None:
    call("nvfp4_debug_wait_timeout", timeout_us, _stream(stream))
