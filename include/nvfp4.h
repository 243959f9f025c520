/*
 * nvfp4.h -- C ABI of the GB300 (sm_103a) NVFP4 block-scaled MoE expert path.
 *
 * NVFP4 tensors: 4-bit E2M1 codes, two per byte (element 2j in the low nibble),
 * one unsigned E4M3 scale per 16 consecutive elements along K, and one FP32
 * global multiplier.  A value decodes as e2m1(code) * e4m3(scale) * global
 * (nvfp4-megamoe-kernel commit log, page 2 = commit efe63ca, single_shot_inference.py:
 * the weight_scale_2 fix, i.e. the NVFP4 dequantisation formula).  Activations carry
 * gs = amax / (6 * 448) as their global multiplier (page 3 = commit 4c6464e, vllm: the
 * activation global-scale passage); weights carry ws2 = weight_scale_2 and nothing else
 * (page 2: the input_scale passage, which keeps the checkpoint input_scale out of the
 * weight side).  A GEMM therefore computes
 * y = (gs * ws2) * sum_k e2m1(a) e4m3(sa) e2m1(b) e4m3(sb)
 * (page 1: the scale-semantics passage, y = (x * scale_a * gsa) @ (w * scale_b * gsb)).
 *
 * Conventions for every entry point:
 *  - Pointers are DEVICE pointers owned by the caller unless stated otherwise;
 *    the library keeps no reference after the call returns and never
 *    allocates device memory.  Calls that need scratch take a caller-owned
 *    workspace (ws, ws_bytes, 256-byte aligned) whose size the matching
 *    *_workspace_bytes query returns; its contents need no initialisation.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream).  Work is enqueued asynchronously; no call synchronises the host
 *    except nvfp4_get_device_error.  Kernels use programmatic dependent launch:
 *    a kernel may start while the previous kernel on the stream finishes, and
 *    reads its inputs only after that kernel completed.  The one exception is
 *    that the GEMMs of nvfp4_linear and of the MoE stages and nvfp4_w4_linear read
 *    the weights and the routing arrays one launch early (the one-token MoE
 *    forward also the token x and its top-k ids and weights).  Those must
 *    therefore be final before the call that opens the chain (nvfp4_linear,
 *    nvfp4_w4_linear, nvfp4_moe_forward or nvfp4_moe_dispatch) is enqueued, which
 *    ordinary stream order gives.
 *  - Kernels on pairs of CTAs (the large products of nvfp4_linear, nvfp4_gemm,
 *    nvfp4_fp8_linear, nvfp4_fp8_gemm, the gated linear and nvfp4_w4_linear of
 *    many tokens) do not run beside one another: across streams, and across the branches of one stream
 *    capture, each waits for the one enqueued before it.  A captured graph that
 *    holds such calls is not ordered against other graphs and streams:
 *    replay it where no other of these calls runs at the same time.
 *  - bf16 tensors are passed as void* to raw bf16 storage (row-major).
 *  - Scale-factor buffers in the "swizzled" tensor-core layout hold
 *    nvfp4_sf_bytes(rows, K) bytes: rows padded to a multiple of 128 and scale
 *    columns (K/16) to a multiple of 4, grouped into 512-byte blocks of
 *    128 rows x 4 columns stored row-group-major; the four scales of row r sit
 *    at byte 16*(r%32) + 4*((r%128)/32) of their block (page 3: the grouped-GEMM
 *    launch contract, A-side scales padded and swizzled).
 *  - Errors: argument problems are detected on the host and returned before
 *    anything is enqueued; nothing throws across the ABI.  A detail string for
 *    the last failing call on the calling thread is available from
 *    nvfp4_last_error_string().  Faults detected on the device (an expert id
 *    out of range, a pipeline wait that timed out) set a per-device flag word
 *    that nvfp4_get_device_error reads.
 *  - Shape rules: K % 64 == 0; GEMM output widths N % 16 == 0 for the dense
 *    linear and GEMM, N % 128 == 0 for the grouped linear and the MoE; all
 *    pointers 16-byte aligned; bf16 row strides a multiple of 8 elements.  Violations
 *    return NVFP4_ERR_UNSUPPORTED_SHAPE or NVFP4_ERR_MISALIGNED.
 */
#ifndef NVFP4_GB300_H
#define NVFP4_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define NVFP4_ABI_VERSION 9

/* Exported symbols: the library builds with hidden visibility by default. */
#if defined(NVFP4_BUILD) && defined(__GNUC__)
#define NVFP4_API __attribute__((visibility("default")))
#else
#define NVFP4_API
#endif

typedef enum nvfp4_status {
  NVFP4_OK = 0,
  NVFP4_ERR_INVALID_ARG = 1,         /* null pointer, negative size, bad enum value     */
  NVFP4_ERR_UNSUPPORTED_SHAPE = 2,   /* K % 64, N % 16 / 128, E or topk out of range    */
  NVFP4_ERR_MISALIGNED = 3,          /* a pointer not 16-byte aligned, bad row stride   */
  NVFP4_ERR_WORKSPACE = 4,           /* ws_bytes below the size the query returns       */
  NVFP4_ERR_CUDA = 5,                /* a CUDA runtime call or launch failed            */
  NVFP4_ERR_DEVICE_FAULT = 6,        /* nvfp4_get_device_error: bad data seen on device */
  NVFP4_ERR_TIMEOUT = 7,             /* nvfp4_get_device_error: a bounded wait ran out  */
  NVFP4_ERR_UNSUPPORTED_DEVICE = 8   /* the current device is not sm_103                */
} nvfp4_status;

/* global-scale modes */
#define NVFP4_GS_DYNAMIC 0  /* compute gs = fl32(amax / 2688) over the whole input, write *gs */
#define NVFP4_GS_STATIC 1   /* read gs from *gs (warm-up calibrated value, page 3)          */

/* scale-factor output layouts of nvfp4_quantize_act */
#define NVFP4_SF_SWIZZLED 0 /* tensor-core layout described above                         */
#define NVFP4_SF_LINEAR 1   /* row-major (M, K/16), the checkpoint layout                 */

/* nvfp4_prepare_weights flags */
#define NVFP4_PREP_PLAIN 0
#define NVFP4_PREP_W13_INTERLEAVE 1 /* rows [0,N/2) gate, [N/2,N) up -> 64 gate + 64 up per 128 */

/* element types of the 16-bit and fp32 operands of the dense feed-forward operators */
#define NVFP4_DT_BF16 0
#define NVFP4_DT_FP16 1
#define NVFP4_DT_FP32 2

/* activations of nvfp4_gated_linear */
#define NVFP4_ACT_SILU 0      /* g / (1 + exp(-g))                                         */
#define NVFP4_ACT_GELU 1      /* g Phi(g), Phi the normal distribution function (erf)      */
#define NVFP4_ACT_GELU_TANH 2 /* g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2           */

/* gates of nvfp4_residual_norm */
#define NVFP4_GATE_NONE 0
#define NVFP4_GATE_CHANNEL 1 /* (groups, K): one value per channel of M / groups rows      */
#define NVFP4_GATE_ROW 2     /* (M): one value per row                                     */

/* device fault flags returned by nvfp4_get_device_error */
#define NVFP4_DEVERR_BAD_EXPERT_ID 1  /* a top-k id outside [0, E); the entry was dropped  */
#define NVFP4_DEVERR_PIPELINE_TIMEOUT 2 /* a GEMM pipeline wait exceeded its limit        */
#define NVFP4_DEVERR_INTERNAL 4         /* a kernel invariant failed (a library bug)      */

NVFP4_API int nvfp4_abi_version(void);
NVFP4_API const char *nvfp4_status_string(nvfp4_status s);
/* Detail of the last non-OK status returned on the calling thread ("" if none). */
NVFP4_API const char *nvfp4_last_error_string(void);

/* Synchronises `stream`, ORs the device fault flags of the current device into
 * *flags and clears them.  Returns NVFP4_ERR_TIMEOUT if the timeout flag is
 * set, NVFP4_ERR_DEVICE_FAULT for any other flag, NVFP4_OK when clear. */
NVFP4_API nvfp4_status nvfp4_get_device_error(void *stream, int32_t *flags);

/* Bytes of a swizzled scale buffer for `rows` rows of K elements. */
NVFP4_API size_t nvfp4_sf_bytes(int64_t rows, int64_t K);

/* ---------------------------------------------------------------- (a) quantize
 * BF16 (M, K) with row stride ldx (elements) -> NVFP4 codes q (M, K/2) and
 * E4M3 block scales sf (swizzled: nvfp4_sf_bytes(M, K) bytes, padding written
 * as 0; linear: M*K/16 bytes).  Per 16-element block b with amax_b = max|x|:
 *   s = fl32(amax_b / fl32(6*gs)), sf = E4M3_rne_satfinite(s),
 *   d = fl32(e4m3(sf) * gs), q_i = E2M1_rne_satfinite(fl32(x_i * fl32(1/d)))
 * with the sign of x_i kept on zero codes, and all codes 0 when d == 0 or 1/d
 * overflows.  gs_mode NVFP4_GS_DYNAMIC computes gs = fl32(amax / 2688) over
 * all M*K elements (two launches: block-max partials, then quantize) and
 * stores it to *gs; NVFP4_GS_STATIC reads *gs.  Workspace: amax partials.
 * With M == 0 only gs is used (dynamic mode writes 0); x, q and sf may be NULL. */
NVFP4_API size_t nvfp4_quantize_workspace_bytes(int64_t M, int64_t K);
NVFP4_API nvfp4_status nvfp4_quantize_act(const void *x, int64_t M, int64_t K, int64_t ldx, int gs_mode,
                                float *gs, uint8_t *q, uint8_t *sf, int sf_layout, void *ws,
                                size_t ws_bytes, void *stream);

/* -------------------------------------------------- RMSNorm -> quantize
 * RMSNorm feeding the activation quantiser (the fused "P4" path of page 1 = commit
 * 1121cd7, single_shot_inference.py: the fused-RMSNorm A/B passage, whose harness compares
 * x_normed, the global scale, the FP4 data and the GEMM outputs of the fused and unfused
 * paths).  Per row r:
 *   inv_r = 1 / sqrt(fl32(sum_k x^2) / K + eps)        (correctly rounded sqrt, divide)
 *   x_normed[r,k] = bf16(fl32(fl32(x[r,k] * inv_r) * gamma[k]))
 * gamma is a bf16 vector of K.  nvfp4_rmsnorm writes x_normed (M, K) bf16 (the unfused
 * path; quantise it with nvfp4_quantize_act).  nvfp4_rmsnorm_quantize quantises x_normed
 * without a round trip through memory, with the same arguments and results as
 * nvfp4_quantize_act applied to nvfp4_rmsnorm's output (codes, scales and dynamic gs
 * bit-identical); x_normed, if not NULL, also receives the normalised rows.  Two launches.
 * Workspace: amax partials and the per-row inv_r. */
NVFP4_API size_t nvfp4_rmsnorm_quantize_workspace_bytes(int64_t M, int64_t K);
NVFP4_API nvfp4_status nvfp4_rmsnorm(const void *x, int64_t M, int64_t K, int64_t ldx, const void *gamma,
                                     float eps, void *y, void *stream);
NVFP4_API nvfp4_status nvfp4_rmsnorm_quantize(const void *x, int64_t M, int64_t K, int64_t ldx,
                                              const void *gamma, float eps, int gs_mode, float *gs,
                                              uint8_t *q, uint8_t *sf, int sf_layout, void *x_normed,
                                              void *ws, size_t ws_bytes, void *stream);

/* ------------------------------------------------------------ weight prepare
 * Checkpoint-layout weights of G groups (experts): codes w (G, N, K/2) and
 * row-major E4M3 scales sf (G, N, K/16) used as stored, no transpose (page 2: the
 * checkpoint-layout fix, N-major codes and untransposed scales).  Writes w_out
 * (nvfp4_prepared_weight_bytes(G, N, K) bytes) and sf_out (G blocks of
 * nvfp4_sf_bytes(N, K)).  The prepared codes are tile-major: for group g, 128-row tile t
 * and 128-byte column slab s of the K/2 code bytes, block ((g * N/128 + t) * S + s),
 * S = ceil(K/256), holds the tile's 128 rows x 128 bytes contiguously (row r at byte
 * 128 r of the 16 KiB block); slab bytes past K/2 are zero codes.  A GEMM stage reads one
 * such block.  NVFP4_PREP_W13_INTERLEAVE reorders the rows of a fused gate/up projection so
 * that every 128-row tile holds 64 gate rows followed by the 64 matching up rows.
 * K % 64 == 0, N % 128 == 0; with G == 1 and no interleave N % 16 == 0 suffices, the
 * last tile's rows from N on then being zero codes and zero scales (sf_out holds
 * nvfp4_sf_bytes(N, K) bytes, which covers them).  Run once at load time; w and w_out
 * must not overlap.
 * Every w / w13 / w2 / sh_* weight argument below is such a prepared buffer. */
NVFP4_API size_t nvfp4_prepared_weight_bytes(int64_t G, int64_t N, int64_t K);
NVFP4_API nvfp4_status nvfp4_prepare_weights(const uint8_t *w, const uint8_t *sf, int64_t G, int64_t N,
                                   int64_t K, int flags, uint8_t *w_out, uint8_t *sf_out,
                                   void *stream);

/* ------------------------------------------------------------ (e) dense linear
 * y (M, N) bf16 = alpha * deq(xq) @ deq(W)^T with alpha = gs * ws2, where xq is
 * x (M, K) bf16 quantised at run time (gs_mode as for nvfp4_quantize_act,
 * *gs written in dynamic mode) and W is a prepared (N, K/2) + swizzled sf
 * weight with device scalar ws2 (Nvfp4Linear, page 2: the ws2-folding fixes).
 * K % 64 == 0, N % 16 == 0 (an N that is not a multiple of 128 ends in a partial tile of
 * the prepared weight; only the first N output columns are written).  Workspace:
 * quantised x + scales + partials. */
NVFP4_API size_t nvfp4_linear_workspace_bytes(int64_t M, int64_t K);
NVFP4_API nvfp4_status nvfp4_linear(const void *x, int64_t M, int64_t K, int64_t N, const uint8_t *w,
                          const uint8_t *w_sf, const float *ws2, int gs_mode, float *gs, void *y,
                          void *ws, size_t ws_bytes, void *stream);

/* Dense linear that allocates nothing and takes no workspace.  (No counterpart
 * on the pages: this entry point exists for callers, not for the method.)
 *
 * Some callers cannot allocate device memory at the point where they run the
 * linear.  Examples are a plugin inside a host inference engine that owns all
 * device memory and forbids allocation while it enqueues work, or a serving
 * loop that reserved a fixed memory budget at start-up and must not touch an
 * allocator per request.  Such a caller may also have no workspace to lend.
 *
 * This variant computes exactly what nvfp4_linear computes, with the same
 * arguments minus (ws, ws_bytes).  Its scratch (the quantised activations, their
 * scales and the amax partials) lives in one file-scope device array of
 * NVFP4_LINEAR_NOALLOC_MAX_BYTES bytes.  Every GPU that loads the library
 * holds that array until the process exits.
 *  - Limit: nvfp4_linear_workspace_bytes(M, K) must not exceed the array size.
 *    For K = 7168 that is M <= 1025; for K = 1536 it is M <= 4848.  Larger
 *    calls return NVFP4_ERR_WORKSPACE before anything is enqueued.
 *  - Set-up: the first call on each device resolves the array's device
 *    address, with that device current.  Make that first call before any
 *    stream capture begins.
 *  - Sharing: all calls on a device use the same array.  It keeps the contents
 *    of the last call, and nothing in it needs to start at zero, because every
 *    byte the GEMM reads is rewritten by the call's own quantise step.  Calls
 *    that overlap on the GPU (different streams without ordering between
 *    them) race on the array and give wrong results: serialise them.
 *  - It calls no cudaMalloc, cudaFree or allocating library routine. */
#define NVFP4_LINEAR_NOALLOC_MAX_BYTES (4u << 20)
NVFP4_API nvfp4_status nvfp4_linear_noalloc(const void *x, int64_t M, int64_t K, int64_t N,
                                            const uint8_t *w, const uint8_t *w_sf,
                                            const float *ws2, int gs_mode, float *gs, void *y,
                                            void *stream);

/* GEMM alone on already-quantised activations: xq (M, K/2) codes with
 * swizzled scales xsf (nvfp4_sf_bytes(M, K)) and device scalar gs; W and ws2
 * as for nvfp4_linear.  y (M, N) bf16. */
NVFP4_API nvfp4_status nvfp4_gemm(const uint8_t *xq, const uint8_t *xsf, const float *gs, int64_t M,
                        int64_t K, int64_t N, const uint8_t *w, const uint8_t *w_sf,
                        const float *ws2, void *y, void *stream);

/* ----------------------------------------------------- fixed-group linear
 * The input features of x (M, G*K) bf16 split into G equal groups of K; group g
 * multiplies its K columns by its own NVFP4 weight W_g (N, K/2) with ws2[g]:
 *   y[:, g*N:(g+1)*N] = (gs * ws2[g]) * deq(xq[:, g*K:(g+1)*K]) @ deq(W_g)^T
 * with one activation gs over all of x (gs_mode as for nvfp4_quantize_act).
 * This is the grouped o-projection of page 3 (the wo_a o-projection passage: a per-group
 * BMM with in_features 4096; the ScaledGroupedGemm passage: an NVFP4 grouped linear with
 * n_local_groups = 8).  w is
 * (G, N, K/2) prepared with NVFP4_PREP_PLAIN and w_sf G blocks of
 * nvfp4_sf_bytes(N, K); ws2 (G) fp32; y (M, G*N) bf16.  K % 64 == 0, N % 128 == 0. */
NVFP4_API size_t nvfp4_grouped_linear_workspace_bytes(int64_t M, int64_t G, int64_t K);
NVFP4_API nvfp4_status nvfp4_grouped_linear(const void *x, int64_t M, int64_t G, int64_t K, int64_t N,
                                            const uint8_t *w, const uint8_t *w_sf, const float *ws2,
                                            int gs_mode, float *gs, void *y, void *ws,
                                            size_t ws_bytes, void *stream);

/* --------------------------------------------------------------- router gate
 * The dense router of page 1 (the router-gate FP8 round-trip passage): the NVFP4 gate
 * weight (E, H/2) codes with row-major scales (E, H/16) and device scalar ws2 is
 * dequantised to bf16, quantised to FP8-E4M3 with one per-tensor scale s = amax / 448 and
 * dequantised back to bf16 (nvfp4_router_prepare, once):
 *   w = bf16(fl32(fl32(e2m1 * e4m3) * ws2)),  q = E4M3(fl32(w * fl32(1/s))),
 *   wg = bf16(fl32(e4m3(q) * s))                       (wg all zero when s == 0)
 * Per call (nvfp4_router): logits = x (T, H) bf16 @ wg^T in fp32, softmax over the E
 * experts, the topk largest probabilities (lower expert id first on ties) as ids (T, topk)
 * int32 and weights (T, topk) fp32 renormalised to sum 1 -- the inputs of the routing
 * stage.  The logits run on the tensor cores split over H; the workspace
 * (nvfp4_router_workspace_bytes, always required) holds the splits' fp32 partials, which
 * are summed in a fixed order, so repeated calls give identical logits.  logits (T, E) fp32,
 * if not NULL, receives the summed logits.  E <= 1024, topk <= min(32, E), H % 64 == 0,
 * T and H below 2^24.  Two launches. */
NVFP4_API size_t nvfp4_router_prepare_workspace_bytes(int64_t E, int64_t H);
NVFP4_API nvfp4_status nvfp4_router_prepare(const uint8_t *w, const uint8_t *w_sf, const float *ws2, int64_t E,
                                            int64_t H, void *wg, void *ws, size_t ws_bytes, void *stream);
NVFP4_API size_t nvfp4_router_workspace_bytes(int64_t T, int64_t E);
NVFP4_API nvfp4_status nvfp4_router(const void *x, int64_t T, int64_t H, const void *wg, int64_t E, int topk,
                                    int32_t *ids, float *weights, float *logits, void *ws, size_t ws_bytes,
                                    void *stream);

/* -------------------------------------------------------------- (b) routing
 * Groups the T*topk flat entries f = t*topk + j of ids (T, topk) int32 by
 * expert: counts[e] (E), offsets (E+1, exclusive prefix sum, int32 as the
 * grouped GEMM wants: page 3, the grouped-GEMM launch contract),
 * sorted_idx (T*topk) = the flat indices ordered by expert, increasing f
 * within an expert, and inv_idx (T*topk) = position of f in sorted_idx.
 * Ids outside [0, E) are dropped (inv_idx = -1) and raise
 * NVFP4_DEVERR_BAD_EXPERT_ID.  1 <= E <= 1024, 1 <= topk <= 32. */
NVFP4_API nvfp4_status nvfp4_moe_route(const int32_t *ids, int64_t T, int topk, int64_t E,
                             int32_t *counts, int32_t *offsets, int32_t *sorted_idx,
                             int32_t *inv_idx, void *stream);

/* ---------------------------------------------------------------- MoE layer
 * Routed experts e in [0, E) plus an optional always-active shared expert
 * (group E).  Weights are prepared with nvfp4_prepare_weights:
 *   w13 (E, 2I, H/2) + sf, NVFP4_PREP_W13_INTERLEAVE (checkpoint rows [0,I)
 *       gate, [I,2I) up), w13_ws2 (E) fp32;
 *   w2  (E, H, I/2) + sf, NVFP4_PREP_PLAIN, w2_ws2 (E) fp32;
 *   sh_w13 / sh_w2 the same for one expert, sh_ws2 = {w13 ws2, w2 ws2};
 *   pass sh_w13 == NULL for no shared expert.
 * For every token t:
 *   y[t] = sum_j topk_w[t,j] * E_{ids[t,j]}(x[t]) + E_shared(x[t]),
 *   E_e(x) = W2_e . requant(SiLU(gate_e(xq)) * up_e(xq); a2_gs[e])
 * with xq = x quantised with one global scale over all T tokens (a1_gs_mode as
 * above, *a1_gs written in dynamic mode) and a2_gs (E+1 entries, last = shared
 * expert) the static global scales of the re-quantised intermediate h
 * (warm-up calibrated, page 3: the warm-up calibration passage).
 * y (T, H) bf16; the output width is H (page 3: the MoE shape-rules passage).  H % 128 == 0, I % 64 == 0.
 * nvfp4_moe_forward with one token (T = 1, topk <= 8, H <= 7168) runs as routing, one GEMM
 * launch and the conversion of y: the GEMM CTAs quantise the token themselves, take their
 * tiles from the ids and add each tile's share of the down projection (its 64 columns of
 * the re-quantised h times that K step of w2) into the fp32 accumulator; the workspace's xq,
 * xsf and amax_partials are then left untouched.  The re-quantised h rows (hq, hsf) are the
 * ones the stage-by-stage calls produce; y agrees within fp32 summation order. */
typedef struct nvfp4_moe_ws_layout {
  /* byte offsets into the workspace */
  size_t counts;        /* int32 [G]        rows per group (G = E + has_shared)     */
  size_t offsets;       /* int32 [G+1]      exclusive scan of counts                 */
  size_t pad_offsets;   /* int32 [G+1]      exclusive scan of counts rounded to 128  */
  size_t tile_offsets;  /* int32 [G+1]      exclusive scan of ceil(counts / R), R the
                           m-tile height: 32 when T <= 128, else 128                */
  size_t sorted_idx;    /* int32 [T*topk]                                            */
  size_t inv_idx;       /* int32 [T*topk]                                            */
  size_t dest_rows;     /* int32 [T*topk]   permuted row of each flat entry (-1 dropped) */
  size_t tile_table;    /* int32x4 [rows_capacity/32] per R-row tile of the permuted
                           buffers, in tile order: group, tile index inside the group
                           (bit 30 set when the group spans several tiles), live rows
                           (1..R), first permuted row                                */
  size_t amax_partials; /* uint32 [1024]    block maxima of |x| as bf16 bits         */
  size_t xq;            /* uint8 [rows_capacity, H/2]  x quantised, permuted rows    */
  size_t xsf;           /* uint8 nvfp4_sf_bytes(rows_capacity, H)                    */
  size_t hq;            /* uint8 [rows_capacity, I/2]  h re-quantised                */
  size_t hsf;           /* uint8 nvfp4_sf_bytes(rows_capacity, I)                    */
  size_t y_acc;         /* float [T, H]     fp32 accumulator of the scatter-add      */
  size_t total;         /* bytes                                                     */
  int64_t rows_capacity; /* padded-row capacity of the permuted buffers              */
  /* row of group g, segment row i in xq/xsf/hq/hsf: pad_offsets[g] + i; routed
   * segment row i of expert e holds flat entry sorted_idx[offsets[e] + i];
   * shared segment row i holds token i. */
} nvfp4_moe_ws_layout;

NVFP4_API nvfp4_status nvfp4_moe_workspace_layout(int64_t T, int64_t H, int64_t I, int64_t E, int topk,
                                        int has_shared, nvfp4_moe_ws_layout *out);
NVFP4_API size_t nvfp4_moe_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t E, int topk,
                                 int has_shared);

NVFP4_API nvfp4_status nvfp4_moe_forward(const void *x, int64_t T, int64_t H, int64_t I, int64_t E,
                               int topk, const int32_t *topk_ids, const float *topk_w,
                               const uint8_t *w13, const uint8_t *w13_sf, const float *w13_ws2,
                               const uint8_t *w2, const uint8_t *w2_sf, const float *w2_ws2,
                               const uint8_t *sh_w13, const uint8_t *sh_w13_sf,
                               const uint8_t *sh_w2, const uint8_t *sh_w2_sf,
                               const float *sh_ws2, int a1_gs_mode, float *a1_gs,
                               const float *a2_gs, void *y, void *ws, size_t ws_bytes,
                               void *stream);

/* The four stages nvfp4_moe_forward enqueues, exposed for stage-wise checks
 * and timing.  Same arguments as nvfp4_moe_forward; they communicate through
 * the workspace (layout above) and must run in this order on one stream. */

/* (a)+(b): routing, global scale, quantisation of x into the permuted rows,
 * zeroing of the fp32 accumulator.  Three launches. */
NVFP4_API nvfp4_status nvfp4_moe_dispatch(const void *x, int64_t T, int64_t H, int64_t I, int64_t E,
                                int topk, const int32_t *topk_ids, int has_shared,
                                int a1_gs_mode, float *a1_gs, void *ws, size_t ws_bytes,
                                void *stream);
/* (c): grouped w13 GEMM, SiLU(gate)*up, NVFP4 re-quantisation into hq/hsf.
 * h_debug, if not NULL, receives the fp32 h rows (rows_capacity, I). */
NVFP4_API nvfp4_status nvfp4_moe_w13(int64_t T, int64_t H, int64_t I, int64_t E, int topk,
                           const uint8_t *w13, const uint8_t *w13_sf, const float *w13_ws2,
                           const uint8_t *sh_w13, const uint8_t *sh_w13_sf, const float *sh_ws2,
                           const float *a1_gs, const float *a2_gs, float *h_debug, void *ws,
                           size_t ws_bytes, void *stream);
/* (d): grouped w2 GEMM with the top-k weighted fp32 scatter-add into y_acc. */
NVFP4_API nvfp4_status nvfp4_moe_w2(int64_t T, int64_t H, int64_t I, int64_t E, int topk,
                          const float *topk_w, const uint8_t *w2, const uint8_t *w2_sf,
                          const float *w2_ws2, const uint8_t *sh_w2, const uint8_t *sh_w2_sf,
                          const float *sh_ws2, const float *a2_gs, void *ws, size_t ws_bytes,
                          void *stream);
/* y (T, H) bf16 = round-to-nearest-even(y_acc). */
NVFP4_API nvfp4_status nvfp4_moe_finalize(int64_t T, int64_t H, int64_t I, int64_t E, int topk,
                                int has_shared, void *y, void *ws, size_t ws_bytes,
                                void *stream);

/* ============================================================================
 * Dense feed-forward operators around the experts: an 8-bit block-scaled linear, a gated
 * linear with its gradients, and the norms, gate and residual sum between two blocks with
 * their gradients.  The conventions above hold (device pointers, no allocation, caller's
 * workspace, programmatic dependent launch, 16-byte aligned pointers); element types are
 * given by NVFP4_DT_*.  What a call writes (outputs, workspace) overlaps neither an input nor anything
 * else it writes, unless the call says so: refused with NVFP4_ERR_INVALID_ARG (of strided rows the whole
 * range from the first element to the last counts).  M, N, K, T, H
 * and I are below 2^24, a product of two of them below 2^40.
 * ============================================================================ */

/* ------------------------------------------- FP8 block-scaled linear (128)
 * e4m3 operands with fp32 scales: one per 128 consecutive K elements of a row of x, one per
 * 128 x 128 block of W (the last block of a row or column may be partial).
 *   s = fl32(max |x| / 448) over the block, q = e4m3_rne_satfinite(fl32(x / s)), q = 0 if s == 0
 *   y[m, n] = sum_b xs[b, m] w_s[n / 128, b] sum_{k in b} q[m, k] w[n, k]       (fp32 sums)
 * A block that holds a NaN or an infinity makes every output of its rows NaN.  xs w_s is formed in
 * fp32 first: below 2^-126 (activations of 1e-32 or less with weights of about 1) it loses bits, and
 * above 2^128 it is infinite.
 * x (M, K), row stride ldx (a multiple of 8), bf16 or fp16; q (M, K) codes, contiguous;
 * xs (ceil(K / 128), lds) fp32, xs[b * lds + m], lds >= M a multiple of 4 (every row,
 * the last included, is readable up to M rounded up to 4; entries m >= M are not written and do not
 * matter); w (N, K) codes and w_s (ceil(N / 128), ceil(K / 128)), both
 * row-major as checkpoints store them: no preparation.  y (M, N) contiguous in `dtype`.
 * K % 16 == 0; any N; K % 16 == 0 for the weight quantiser too (ldw a multiple of 8). */
NVFP4_API nvfp4_status nvfp4_fp8_quantize_act(const void *x, int dtype, int64_t M, int64_t K, int64_t ldx,
                                              uint8_t *q, float *xs, int64_t lds, void *stream);
NVFP4_API nvfp4_status nvfp4_fp8_quantize_weight(const void *w, int dtype, int64_t N, int64_t K, int64_t ldw,
                                                 uint8_t *q, float *w_s, void *stream);
NVFP4_API nvfp4_status nvfp4_fp8_gemm(const uint8_t *xq, const float *xs, int64_t lds, int64_t M, int64_t K,
                                      int64_t N, const uint8_t *w, const float *w_s, int dtype, void *y,
                                      void *stream);
/* The quantiser and the product in one call, with the two calls' results bit for bit; the workspace
 * holds the codes and scales.  With few rows (M <= 16, or up to 64 of a small product) the product
 * quantises x itself: one launch; up to 16 rows the workspace's size is 0. */
NVFP4_API size_t nvfp4_fp8_linear_workspace_bytes(int64_t M, int64_t K);
NVFP4_API nvfp4_status nvfp4_fp8_linear(const void *x, int dtype, int64_t M, int64_t K, int64_t ldx, int64_t N,
                                        const uint8_t *w, const float *w_s, void *y, void *ws, size_t ws_bytes,
                                        void *stream);

/* ------------------------------------------------------------ gated linear
 * h = act(x Wg^T) * (x Wu^T): both projections, the activation and the product in one kernel.
 * x (T, H), row stride ldx (a multiple of 8); w_gate and w_up (I, H) contiguous; h (T, I)
 * contiguous; all bf16 or all fp16 (`dtype`).  gu, if not NULL, receives the fp32
 * pre-activations (T, 2I), g in columns [0, I) and u in [I, 2I), 32-byte aligned: the input of the
 * backward.
 * H % 8 == 0, I % 8 == 0. */
NVFP4_API nvfp4_status nvfp4_gated_linear(const void *x, int dtype, int64_t T, int64_t H, int64_t ldx, int64_t I,
                                          const void *w_gate, const void *w_up, int act, void *h, float *gu,
                                          void *stream);
/* Gradients of h: dg = dh u act'(g) and du = dh act(g), rounded to `dtype`'s precision, then
 *   dx = dg Wg + du Wu (T, H),  dw_gate = dg^T x (I, H),  dw_up = du^T x (I, H)
 * with fp32 sums, contiguous, in `dtype`.  For fp16 the products take dg and du times a power of two, divided out of
 * the sums, that puts the largest finite magnitude of both between 2^14 and 2^15: they neither overflow nor lose bits
 * but where they are below 2^-28 of that one.  dx may be NULL, and dw_gate and dw_up may both be
 * NULL: that product is then left out.  dh (T, I) has row stride lddh (a multiple of 8).
 * With T == 0 the weight gradients are zero.  Workspace: [dg | du], and 4352 bytes more for fp16 (the size by dtype;
 * the query without one is bf16's). */
NVFP4_API size_t nvfp4_gated_linear_backward_workspace_bytes(int64_t T, int64_t I);
NVFP4_API size_t nvfp4_gated_linear_backward_workspace_bytes_dt(int64_t T, int64_t I, int dtype);
NVFP4_API nvfp4_status nvfp4_gated_linear_backward(const void *dh, int64_t lddh, const void *x, int64_t ldx,
                                                   int dtype, int64_t T, int64_t H, int64_t I,
                                                   const void *w_gate, const void *w_up, int act, const float *gu,
                                                   void *dx, void *dw_gate, void *dw_up, void *ws,
                                                   size_t ws_bytes, void *stream);

/* ----------------------------------------------------------- residual norm
 * The boundary between two blocks of a layer: the norm after the block, its gate and residual
 * scale, the residual sum, and the norm before the next block.  Per row, in fp32:
 *   n = f rstd(f) gamma_after        (n = f if gamma_after is NULL)
 *   r_out = r + scale gate n
 *   y = r_out rstd(r_out) gamma_before   (from r_out before its rounding; none if NULL)
 * with rstd(v) = 1 / sqrt(mean(v^2) + eps).  f (M, K) with row stride ldf, gammas (K) and the gate
 * in `dtype` (bf16 or fp16); r (M, K) with row stride ldr and r_out (M, K) contiguous in
 * `r_dtype`: `dtype` or fp32.  gate_kind NVFP4_GATE_CHANNEL: gate (gate_groups, K) contiguous, row
 * m uses gate[m / (M / gate_groups)], M % gate_groups == 0; NVFP4_GATE_ROW: gate (M).
 * y (M, K) contiguous in `dtype`.  stats, if not NULL: fp32 (M, 2) = rstd(f), rstd(r_out) (0 where
 * a norm is absent), the input of the backward.  r_out may be r (same stride K) if stats is NULL, since
 * the backward reads r, and else overlaps neither r nor f.
 * K % 8 == 0, K <= 16384; row strides a multiple of 8. */
NVFP4_API nvfp4_status nvfp4_residual_norm(const void *f, int dtype, const void *r, int r_dtype, int64_t M,
                                           int64_t K, int64_t ldf, int64_t ldr, const void *gamma_after,
                                           const void *gate, int gate_kind, int64_t gate_groups, float scale,
                                           const void *gamma_before, float eps, void *r_out, void *y,
                                           float *stats, void *stream);
/* The same with y in 8 bits, as nvfp4_fp8_gemm reads it: e4m3 codes q (M, K), contiguous, and xs (ceil(K / 128), lds)
 * with xs[b * lds + m] = fl32(max |y| / 448) over columns 128 b .. 128 b + 127 of row m and q = e4m3(y / xs) (0 where xs is
 * 0), from y in fp32: rounded once, so the codes can differ from those of nvfp4_fp8_quantize_act on the
 * 16-bit y, which is rounded twice.  The quotient is within a step of fp32.  A block that holds a NaN or an infinity
 * has such a scale.  y, if not NULL, also receives the 16-bit output; r_out, y and stats are those of nvfp4_residual_norm
 * bit for bit (the backward of y is nvfp4_residual_norm_backward's; the rounding to 8 bits has no gradient of its own).
 * gamma_before is required; K % 16 == 0; lds >= M, a multiple of 4 (entries m >= M are not written). */
NVFP4_API nvfp4_status nvfp4_residual_norm_fp8(const void *f, int dtype, const void *r, int r_dtype, int64_t M,
                                               int64_t K, int64_t ldf, int64_t ldr, const void *gamma_after,
                                               const void *gate, int gate_kind, int64_t gate_groups, float scale,
                                               const void *gamma_before, float eps, void *r_out, uint8_t *q, float *xs,
                                               int64_t lds, void *y, float *stats, void *stream);
/* Gradients, from the gradients dr_out of r_out (r_dtype, row stride lddr) and dy of y (dtype, row
 * stride lddy); either may be NULL (zero).  f, r, the parameters and stats are the forward's.
 * df (M, K) in dtype, dr (M, K) in r_dtype, contiguous; dgamma_after (K), dgamma_before (K) and
 * dgate (the gate's shape) in fp32, each sum over rows in a fixed order; each of the three may be
 * NULL, and has to be where its parameter is absent.  With M == 0 the parameter gradients are zero. */
NVFP4_API size_t nvfp4_residual_norm_backward_workspace_bytes(int64_t M, int64_t K, int64_t gate_groups,
                                                              int r_dtype);
NVFP4_API nvfp4_status nvfp4_residual_norm_backward(const void *dr_out, int64_t lddr, const void *dy, int64_t lddy,
                                                    const void *f, int dtype, const void *r, int r_dtype,
                                                    int64_t M, int64_t K, int64_t ldf, int64_t ldr,
                                                    const float *stats, const void *gamma_after, const void *gate,
                                                    int gate_kind, int64_t gate_groups, float scale,
                                                    const void *gamma_before, void *df, void *dr,
                                                    float *dgamma_after, float *dgate, float *dgamma_before,
                                                    void *ws, size_t ws_bytes, void *stream);

/* ============================================================================
 * 4-bit integer weights with group scales, and 16-bit activations: for inference.  A checkpoint stores, for each row
 * of a matrix (N, K), codes c of 4 bits (two per byte, element 2 j in the low half; K / 2 bytes), and for each `group` (32,
 * 64 or 128) consecutive K elements, the last group of a row may be partial, a scale s in `dtype` and, optionally, a
 * zero point z (one byte, of which the low four bits count, so that a file that stores z - 1 has to be raised by its
 * reader and its 15 stands for no z; 8 without zero points).  A weight is (c - z) s.
 * The conventions of the dense operators hold; x (rows, K) has a row stride ldx (a multiple of 8) and is bf16 or fp16
 * (`dtype`), the scales' type; K % 8 == 0.  Weights are never rounded: products with c - z are exact, a group's sum is fp32 (of 2^-7 of its
 * size in bf16, 2^-10 in fp16) and multiplied by its scale in fp32.  A row of x that holds a NaN or an infinity has outputs that are not finite.
 * ============================================================================ */

/* Lays out G matrices for the products below, once, at load time: codes (G, N, K / 2), scales and zeros (G, N,
 * ceil(K / group)), contiguous; out nvfp4_w4_prepared_bytes(G, N, K, group, zeros != NULL, gated) bytes (0: sizes that are not
 * supported).  `gated`: rows [0, N / 2) are a gate projection and [N / 2, N) the up projection of the same outputs (the layout
 * that the mixture-of-experts layer wants of w13), N even.  dtype: the scales' type, which the products must be given too. */
NVFP4_API size_t nvfp4_w4_prepared_bytes(int64_t G, int64_t N, int64_t K, int group, int has_zeros, int gated);
NVFP4_API nvfp4_status nvfp4_w4_prepare(const uint8_t *codes, const void *scales, const uint8_t *zeros, int dtype,
                                        int64_t G, int64_t N, int64_t K, int group, int gated, uint8_t *out,
                                        void *stream);

/* y (M, N) = x (M, K) W^T, contiguous in `dtype`, W prepared without `gated`; any N, any M.  For few tokens the weights are read one
 * launch early, like those of nvfp4_linear, and no workspace is needed; for many it holds the weights' codes in 16 bits
 * and the scales in fp32 (about 2 N K bytes).  The size returned for M rows is enough for every smaller number of rows too. */
NVFP4_API size_t nvfp4_w4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int group);
NVFP4_API nvfp4_status nvfp4_w4_linear(const void *x, int dtype, int64_t M, int64_t K, int64_t ldx, int64_t N,
                                       const uint8_t *w, int group, int has_zeros, void *y, void *ws, size_t ws_bytes,
                                       void *stream);

/* A whole mixture-of-experts layer for a few tokens, in two launches: for every token t
 *   l = x[t] router^T (fp32), ids = the topk largest of l (the lowest expert first among equals),
 *   p = softmax of l over the chosen ones (the softmax over all experts, renormalised),
 *   y[t] = sum_j p_j E_{ids_j}(x[t]) + E_shared(x[t]),  E(x) = W2 h,  h = act(Wg x) * (Wu x) rounded to `dtype`
 * with fp32 sums; h is the operand of a 16-bit product, as in a layer that stores it.  In fp16 a row of h that passes 65504 is
 * held times a power of two: it does not overflow (elements under 2^-28 of its largest lose bits).  x (T, H) with row stride ldx;
 * router (E, H) in `dtype`, contiguous; w13 (E, 2 I, H) prepared with `gated`, w2 (E, H, I) without; sh_w13 and sh_w2 the same for one
 * expert, both NULL without a shared expert; y (T, H) contiguous; act NVFP4_ACT_*.  Sums have a fixed order: repeated calls give
 * identical bits.  T <= 64, topk <= 16, topk <= E <= 1024, T topk <= 512; H and I multiples of 8, at most
 * 16384.  Tokens of one expert share a pass over its weights eight at a time. */
NVFP4_API size_t nvfp4_w4_moe_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t E, int topk, int has_shared);
NVFP4_API nvfp4_status nvfp4_w4_moe(const void *x, int dtype, int64_t T, int64_t H, int64_t ldx, int64_t I, int64_t E,
                                    int topk, const void *router, const uint8_t *w13, const uint8_t *w2,
                                    const uint8_t *sh_w13, const uint8_t *sh_w2, int group, int has_zeros, int act,
                                    void *y, void *ws, size_t ws_bytes, void *stream);

/* ------------------------------------------------------------ diagnostics
 * Runs one CTA that waits on a shared-memory barrier nothing arrives at, with
 * the same bounded-wait helper the GEMM pipeline uses and a limit of
 * timeout_us; it must give up, raise NVFP4_DEVERR_PIPELINE_TIMEOUT and return.
 * Used to test the timeout path without a fault. */
NVFP4_API nvfp4_status nvfp4_debug_wait_timeout(uint32_t timeout_us, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* NVFP4_GB300_H */
