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
# graph: a backward pass is its own call, and those that have one refuse inputs that require grad while
# gradients are recorded (the FP8 linear has none and is for inference, like ``linear``).  An output given as ``out`` and a ``workspace``
# overlap no input and not one another (``residual_norm``'s ``out`` may be r itself).  With ``stream`` given, outputs and scratch are allocated
# for that stream and the inputs are marked as used on it.  Large products of different streams run
# one after the other; a captured graph that holds some is replayed where no other runs at the
# same time (on one stream, or on several that wait for one another).

_DT = {torch.bfloat16: _lib.DT_BF16, torch.float16: _lib.DT_FP16}
_ACT = {"silu": _lib.ACT_SILU, "gelu": _lib.ACT_GELU, "gelu_tanh": _lib.ACT_GELU_TANH}
_CODES = (torch.float8_e4m3fn, torch.uint8)


def _here(stream, *tensors: Optional[torch.Tensor]) -> int:
    """Raw handle of the current stream if the call can run as it stands, -1 if ``_elsewhere`` has to
    switch to the given stream or to the tensors' device first; refuses mixed or CPU tensors."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("tensors on different devices")
    if dev < 0:
        raise ValueError("nvfp4 ops take CUDA tensors only (no CPU fallback)")
    if stream is not None or dev != torch._C._cuda_getDevice():
        return -1
    return torch._C._cuda_getCurrentRawStream(dev)


def _no_graph(*tensors: Optional[torch.Tensor]) -> None:
    """Refuses what would silently cut an autograd graph."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise ValueError("an input requires grad, but this call records no graph: make it under torch.no_grad() "
                                 "and take the gradients from the operator's backward call")


def _elsewhere(stream, tensors, run):
    """``run()`` with the tensors' device current and on ``stream`` (if given), which the tensors are
    marked as used on; outputs and scratch then belong to that stream too."""
    device = next(t for t in tensors if t is not None).device
    with torch.cuda.device(device):
        if stream is None:
            return run()
        if stream.device != device:
            raise ValueError("stream of another device")
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        with torch.cuda.stream(stream):
            return run()


def _kind(x: torch.Tensor, what: str) -> int:
    d = _DT.get(x.dtype)
    if d is None:
        raise ValueError(f"{what} must be bf16 or fp16, got {x.dtype}")
    return d


def _ld(t: torch.Tensor, what: str, rows: int, cols: int, dtype=None) -> int:
    """Row stride of a 2-D tensor of strided rows (a single row's stride does not matter)."""
    if t.shape != (rows, cols) or (dtype is not None and t.dtype != dtype):
        raise ValueError(f"{what} has shape {tuple(t.shape)} and type {t.dtype}, expected ({rows}, {cols}) "
                         f"{dtype if dtype is not None else ''}")
    ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{what}: the elements of a row must be contiguous")
    return ld if rows > 1 else cols


def _size(t: torch.Tensor, what: str):
    """(rows, columns) of a 2-D tensor."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{what} must be 2-D, got {tuple(shape)}")
    return shape


def _whole(t: torch.Tensor, what: str, shape, dtypes) -> int:
    """Data pointer of a contiguous tensor of the given shape and type."""
    if t.shape != shape or t.dtype not in dtypes:
        raise ValueError(f"{what} has shape {tuple(t.shape)} and type {t.dtype}, expected {shape} {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _scratch(workspace: Optional[torch.Tensor], query: str, like: torch.Tensor, *sizes: int):
    """The caller's workspace or a new one of the size that the query returns (None for size 0), and
    its bytes."""
    if workspace is None:
        n = getattr(lib(), query)(*sizes)
        return (torch.empty(n, dtype=torch.uint8, device=like.device) if n else None), n
    n = workspace.numel()
    _whole(workspace, "workspace", (n,), (torch.uint8,))
    return workspace, n


def fp8_quantize_act(x: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """x (M, K) strided rows -> (q (M, K) float8_e4m3fn, s (ceil(K / 128), M) fp32).

    One scale per 128 consecutive K elements of a row, s = max|x| / 448, q = e4m3(x / s).  s is a view
    of rows padded to a multiple of four, as ``fp8_gemm`` wants them.  K % 16 == 0.
    """
    st = _here(stream, x)
    if st < 0:
        return _elsewhere(stream, (x,), lambda: fp8_quantize_act(x))
    M, K = _size(x, "x")
    ld = _ld(x, "x", M, K)
    q = torch.empty(M, K, dtype=torch.float8_e4m3fn, device=x.device)
    lds = (M + 3) // 4 * 4
    s = torch.empty((K + 127) // 128, lds, dtype=torch.float32, device=x.device)
    call("nvfp4_fp8_quantize_act", x.data_ptr(), _kind(x, "x"), M, K, ld, q.data_ptr(), s.data_ptr(), lds, st)
    return q, s[:, :M]


def fp8_quantize_weight(w: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """w (N, K) strided rows -> (q (N, K) float8_e4m3fn, s (ceil(N / 128), ceil(K / 128)) fp32): one
    scale per 128 x 128 block, the layout checkpoints store.  Once, at load time.  K % 16 == 0."""
    st = _here(stream, w)
    if st < 0:
        return _elsewhere(stream, (w,), lambda: fp8_quantize_weight(w))
    N, K = _size(w, "w")
    ld = _ld(w, "w", N, K)
    q = torch.empty(N, K, dtype=torch.float8_e4m3fn, device=w.device)
    s = torch.empty((N + 127) // 128, (K + 127) // 128, dtype=torch.float32, device=w.device)
    call("nvfp4_fp8_quantize_weight", w.data_ptr(), _kind(w, "w"), N, K, ld, q.data_ptr(), s.data_ptr(), st)
    return q, s


def _fp8_weight(w: torch.Tensor, w_s: torch.Tensor, K: int) -> Tuple[int, int, int]:
    N = _size(w, "w")[0]
    return (N, _whole(w, "w", (N, K), _CODES),
            _whole(w_s, "w_s", ((N + 127) // 128, (K + 127) // 128), (torch.float32,)))


def fp8_gemm(xq: torch.Tensor, xs: torch.Tensor, w: torch.Tensor, w_s: torch.Tensor, dtype=torch.bfloat16,
             out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y (M, N) = deq(xq) deq(w)^T of quantised activations (``fp8_quantize_act``) and weights, in
    bf16 or fp16; the scales apply to fp32 sums of one 128-wide K block each."""
    st = _here(stream, xq, xs, w, w_s, out)
    if st < 0:
        return _elsewhere(stream, (xq, xs, w, w_s, out), lambda: fp8_gemm(xq, xs, w, w_s, dtype, out))
    M, K = _size(xq, "xq")
    _size(xs, "xs")
    N, wp, wsp = _fp8_weight(w, w_s, K)
    KB = (K + 127) // 128
    # the stride of a single row, or of empty ones, says nothing
    lds = (M + 3) // 4 * 4 if KB == 1 or M == 0 else xs.stride(0)
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
    st = _here(stream, x, w, w_s, out, workspace)
    if st < 0:
        return _elsewhere(stream, (x, w, w_s, out, workspace), lambda: fp8_linear(x, w, w_s, out, workspace))
    M, K = _size(x, "x")
    ld = _ld(x, "x", M, K)
    N, wp, wsp = _fp8_weight(w, w_s, K)
    if out is not None:
        _whole(out, "out", (M, N), (x.dtype,))
    y = out if out is not None else torch.empty(M, N, dtype=x.dtype, device=x.device)
    ws, ws_bytes = _scratch(workspace, "nvfp4_fp8_linear_workspace_bytes", x, M, K)
    call("nvfp4_fp8_linear", x.data_ptr(), _kind(x, "x"), M, K, ld, N, wp, wsp, y.data_ptr(), _ptr(ws), ws_bytes, st)
    return y


def _gated_args(x, w_gate, w_up, activation):
    if activation not in _ACT:
        raise ValueError(f"activation {activation!r}, expected one of {sorted(_ACT)}")
    T, H = _size(x, "x")
    ld = _ld(x, "x", T, H)
    I = _size(w_gate, "w_gate")[0]
    return (T, H, I, ld, _kind(x, "x"), _whole(w_gate, "w_gate", (I, H), (x.dtype,)),
            _whole(w_up, "w_up", (I, H), (x.dtype,)), _ACT[activation])


def gated_linear(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, activation: str = "silu",
                 save: bool = False, out: Optional[torch.Tensor] = None, stream=None):
    """h (T, I) = act(x w_gate^T) * (x w_up^T): x (T, H) strided rows, weights (I, H), one type.

    ``activation``: "silu", "gelu" (erf) or "gelu_tanh".  With ``save`` returns (h, gu), gu (T, 2I) the
    fp32 pre-activations [g | u] that ``gated_linear_backward`` takes.  H % 8 == 0, I % 8 == 0.
    """
    st = _here(stream, x, w_gate, w_up, out)
    _no_graph(x, w_gate, w_up)
    if st < 0:
        return _elsewhere(stream, (x, w_gate, w_up, out), lambda: gated_linear(x, w_gate, w_up, activation, save, out))
    T, H, I, ld, kind, gp, up, act = _gated_args(x, w_gate, w_up, activation)
    if out is not None:
        _whole(out, "out", (T, I), (x.dtype,))
    h = out if out is not None else torch.empty(T, I, dtype=x.dtype, device=x.device)
    gu = torch.empty(T, 2 * I, dtype=torch.float32, device=x.device) if save else None
    call("nvfp4_gated_linear", x.data_ptr(), kind, T, H, ld, I, gp, up, act, h.data_ptr(), _ptr(gu), st)
    return (h, gu) if save else h


def gated_linear_backward(dh: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
                          gu: torch.Tensor, activation: str = "silu", need_dx: bool = True, need_dw: bool = True,
                          workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients (dx (T, H), dw_gate (I, H), dw_up (I, H)) of ``gated_linear`` from dh (T, I) strided
    rows and the saved gu; those not asked for are None."""
    st = _here(stream, x, dh, w_gate, w_up, gu, workspace)
    _no_graph(x, dh, w_gate, w_up)
    if st < 0:
        return _elsewhere(stream, (x, dh, w_gate, w_up, gu, workspace),
                          lambda: gated_linear_backward(dh, x, w_gate, w_up, gu, activation, need_dx, need_dw, workspace))
    T, H, I, ld, kind, gp, up, act = _gated_args(x, w_gate, w_up, activation)
    lddh = _ld(dh, "dh", T, I, x.dtype)
    gup = _whole(gu, "gu", (T, 2 * I), (torch.float32,))
    dx = torch.empty(T, H, dtype=x.dtype, device=x.device) if need_dx else None
    dwg = torch.empty(I, H, dtype=x.dtype, device=x.device) if need_dw else None
    dwu = torch.empty(I, H, dtype=x.dtype, device=x.device) if need_dw else None
    ws, ws_bytes = _scratch(workspace, "nvfp4_gated_linear_backward_workspace_bytes_dt", x, T, I, kind)
    call("nvfp4_gated_linear_backward", dh.data_ptr(), lddh, x.data_ptr(), ld, kind, T, H, I, gp, up, act, gup,
         _ptr(dx), _ptr(dwg), _ptr(dwu), _ptr(ws), ws_bytes, st)
    return dx, dwg, dwu


def _norm_args(f, r, gamma_after, gate, gamma_before):
    M, K = _size(f, "f")
    ldf, kind = _ld(f, "f", M, K), _kind(f, "f")
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
    if gate.dim() not in (1, 2):
        raise ValueError(f"gate has shape {tuple(gate.shape)}, expected ({K},), (groups, {K}) or ({M}, 1)")
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
    or (M, 1).  ``out`` receives r_out and may be r, but not with ``save``: the backward reads the r that
    would be overwritten.  K % 8 == 0, K <= 16384.
    """
    st = _here(stream, f, r, gamma_after, gate, gamma_before, out)
    _no_graph(f, r, gamma_after, gate, gamma_before)
    if st < 0:
        return _elsewhere(stream, (f, r, gamma_after, gate, gamma_before, out),
                          lambda: residual_norm(f, r, gamma_after, gate, scale, gamma_before, eps, save, out))
    M, K, ldf, ldr, kind, rkind, ga, gp, gkind, groups, gb = _norm_args(f, r, gamma_after, gate, gamma_before)
    if out is not None:
        _whole(out, "out", (M, K), (r.dtype,))
    r_out = out if out is not None else torch.empty(M, K, dtype=r.dtype, device=r.device)
    y = torch.empty(M, K, dtype=f.dtype, device=f.device) if gb is not None else None
    stats = torch.empty(M, 2, dtype=torch.float32, device=f.device) if save else None
    call("nvfp4_residual_norm", f.data_ptr(), kind, r.data_ptr(), rkind, M, K, ldf, ldr, ga, gp, gkind, groups, scale,
         gb, eps, r_out.data_ptr(), _ptr(y), _ptr(stats), st)
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
    st = _here(stream, f, r, dr_out, dy, stats, gamma_after, gate, gamma_before, workspace)
    _no_graph(f, r, dr_out, dy, gamma_after, gate, gamma_before)
    if st < 0:
        return _elsewhere(stream, (f, r, dr_out, dy, stats, gamma_after, gate, gamma_before, workspace),
                          lambda: residual_norm_backward(dr_out, dy, f, r, stats, gamma_after, gate, scale, gamma_before,
                                                         eps, workspace))
    M, K, ldf, ldr, kind, rkind, ga, gp, gkind, groups, gb = _norm_args(f, r, gamma_after, gate, gamma_before)
    if dy is not None and gb is None:
        raise ValueError("dy without gamma_before")
    lddr = K if dr_out is None else _ld(dr_out, "dr_out", M, K, r.dtype)
    lddy = K if dy is None else _ld(dy, "dy", M, K, f.dtype)
    sp = _whole(stats, "stats", (M, 2), (torch.float32,))
    df = torch.empty(M, K, dtype=f.dtype, device=f.device)
    dr = torch.empty(M, K, dtype=r.dtype, device=r.device)

    def grad(p):
        return None if p is None else torch.empty(p.shape, dtype=torch.float32, device=f.device)

    dga, dgate, dgb = grad(gamma_after), grad(gate), grad(gamma_before)
    ws, ws_bytes = _scratch(workspace, "nvfp4_residual_norm_backward_workspace_bytes", f, M, K, max(groups, 1), rkind)
    call("nvfp4_residual_norm_backward", _ptr(dr_out), lddr, _ptr(dy), lddy, f.data_ptr(), kind, r.data_ptr(), rkind,
         M, K, ldf, ldr, sp, ga, gp, gkind, groups, scale, gb, df.data_ptr(), dr.data_ptr(), _ptr(dga), _ptr(dgate),
         _ptr(dgb), _ptr(ws), ws_bytes, st)
    return df, dr, dga, dgate, dgb


# --------------------------------------------------------------------------- diagnostics

def device_error(stream=None) -> Tuple[int, int]:
    """(status, flags) of the device fault word; synchronises the stream and clears the flags."""
    flags = _lib.ctypes.c_int32(0)
    st = lib().nvfp4_get_device_error(_stream(stream), _lib.ctypes.byref(flags))
    return int(st), int(flags.value)


def debug_wait_timeout(timeout_us: int, stream=None) -> None:
    call("nvfp4_debug_wait_timeout", timeout_us, _stream(stream))
