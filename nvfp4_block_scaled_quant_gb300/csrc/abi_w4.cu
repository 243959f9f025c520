// Host side of the C ABI of the operators on 4-bit weights with group scales: argument validation, workspace layout and
// how a product spreads over the GPU.
#include "abi_util.h"
#include "tile_gemm.cuh"
#include "w4.h"

namespace nvfp4 {
namespace {

nvfp4_status check_w4(const char *fn, int dtype, int64_t K, int group) {
  if (!dtype16(dtype)) return fail(NVFP4_ERR_INVALID_ARG, fn, "dtype %d is neither bf16 nor fp16", dtype);
  if (group != 32 && group != 64 && group != 128) return fail(NVFP4_ERR_INVALID_ARG, fn, "group size %d, expected 32, 64 or 128", group);
  if (K % 8) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, fn, "K=%lld must be a multiple of 8", (long long)K);
  return NVFP4_OK;
}

// Bytes of G prepared matrices (N, K).
int64_t prepared_bytes(int64_t G, int64_t N, int64_t K, int group, bool zeros, bool gated) {
  return G * w4_panels(N, gated) * w4_blocks(K) * w4_block_bytes(kW4BlockK / group, zeros);
}

nvfp4_status check_rows(const char *fn, const void *x, int64_t M, int64_t K, int64_t ldx) {
  if (!x && M > 0) return fail(NVFP4_ERR_INVALID_ARG, fn, "x is NULL");
  if (ldx < K || ldx % 8 || ldx >= kMaxDim * 16)
    return fail(NVFP4_ERR_MISALIGNED, fn, "row stride %lld must be >= %lld and a multiple of 8", (long long)ldx, (long long)K);
  if (!aligned(x, 16)) return fail(NVFP4_ERR_MISALIGNED, fn, "x must be 16-byte aligned");
  return NVFP4_OK;
}

// Clusters along K for `ctas` CTAs per split: waves of two CTAs per SM, each as long as a warp's K blocks and a fixed part
// (start, sums over the cluster) of about two.
int stream_splits(int64_t ctas, int blocks, int sms) {
  int best = 1;
  int64_t best_time = 0;
  for (int s = 1; s <= 8 && s <= blocks; ++s) {
    const int64_t waves = (ctas * s + 2 * sms - 1) / (2 * sms), rank = (blocks + s - 1) / s;
    const int64_t time = waves * ((rank + 7) / 8 + 2);
    if (best_time == 0 || time < best_time) best_time = time, best = s;
  }
  return best;
}

// Estimated times in ns that choose between the kernels, their tiles and splits.  The coefficients were fitted to times on a
// GB300 over 32 to 1024 tokens and six (K, N) between 512 x 512 and 7168 x 7168, every choice of each measured (the chosen one is
// 0.1% slower than the best on average); they rank the choices, nothing else depends on them.  Groups of 64 and 32 take longer
// where each group's sums pass through registers.
constexpr int64_t kTcStart[3] = {5200, 6100, 7900}, kTcBlock[3] = {470, 620, 720};  // by tokens of a tile: 32, 64, 128
constexpr int64_t kTileStart = 5400, kTileEnd[2] = {2200, 1500}, kTileBlock[2] = {272, 205};   // 256 and 128 columns; 64 K

// How w4_tc_kernel covers M tokens: tiles of `tok`, clusters of `splits` CTAs along K, one CTA to an SM.
constexpr int kTcClusters[4] = {152, 76, 46, 36};  // of 1 to 4 CTAs that a GB300 holds at once
constexpr int kPlanPairs = 76;                     // of CTAs
struct TcPlan {
  int tok, splits;
  int64_t time;
};
TcPlan tc_plan(int64_t M, int64_t N, int64_t K, int group) {
  TcPlan p = {32, 1, 0};
  int size = 0;
  while (p.tok < 128 && p.tok < M) p.tok *= 2, ++size;
  const int64_t tiles = (N + 127) / 128 * ((M + p.tok - 1) / p.tok), blocks = w4_blocks(K);
  const int64_t block = kTcBlock[size] * (group == 32 ? 174 : group == 64 ? 110 : 100) / 100;
  for (int s = 1; s <= 4 && s <= blocks; ++s) {
    const int64_t waves = (tiles + kTcClusters[s - 1] - 1) / kTcClusters[s - 1];
    const int64_t time = waves * ((blocks + s - 1) / s * block + kTcStart[size]);
    if (p.time == 0 || time < p.time) p.time = time, p.splits = s;
  }
  return p;
}

// The pair GEMM behind the expansion: columns (tokens) of a tile.
struct PairPlan {
  int cols;
  int64_t time;
};
PairPlan pair_plan(int64_t M, int64_t N, int64_t K, int group) {
  PairPlan p = {256, 0};
  const int64_t expand = N * K / 2640;  // 2.5 bytes a weight
  for (int i = 0; i < 2; ++i) {
    const int cols = i ? 128 : 256;
    const int64_t tiles = (N + kTRows - 1) / kTRows * ((M + cols - 1) / cols), waves = (tiles + kPlanPairs - 1) / kPlanPairs;
    const int64_t block = kTileBlock[i] * (group == 32 ? 27 : group == 64 ? 14 : 10) / 10;
    const int64_t time = kTileStart + expand + waves * ((K + 63) / 64 * block + kTileEnd[i]);
    if (p.time == 0 || time < p.time) p = {cols, time};
  }
  return p;
}

// Which kernel takes M tokens.  Up to 16 the weight-streaming one is faster whatever the sizes (16 tokens of 7168 -> 7168 13.6
// against 20 us, 1536 -> 16384 7.2 against 11).  Above, the estimates decide, from sizes alone for the full GPU, since they
// also size the workspace, which is asked for without a device; a choice made for 152 SMs is right on fewer, if not the fastest.
constexpr int64_t kStreamMaxTokens = 16;
constexpr int64_t kTcMaxTokens = int64_t(65535) * 128;  // the grid's second dimension
bool takes_pairs(int64_t M, int64_t N, int64_t K, int group) {
  if (M > kTcMaxTokens) return true;
  return M > kStreamMaxTokens && pair_plan(M, N, K, group).time < tc_plan(M, N, K, group).time;
}

// ... of any number of rows up to M.  The estimates are steps of M, so that the choice can go back and forth as M grows (12288 x 4096
// in groups of 32: pairs for 129 to 256 rows, not up to 384, again beyond); a step ends at each of the numbers tried.  From
// 8192 rows on, where x and y outweigh the weights of any product that has not taken pairs by then, the answer is yes.
bool may_take_pairs(int64_t M, int64_t N, int64_t K, int group) {
  if (M <= kStreamMaxTokens) return false;
  for (int64_t m = 32; m < 8192; m += m < 128 ? m : 128) {
    if (takes_pairs(m, N, K, group)) return true;
    if (m >= M) return false;
  }
  return true;
}

// For the pair GEMM: where the written-out weights and their scales are in the workspace.
struct LinearWs {
  size_t scales, total;
  int64_t lds;
};
LinearWs linear_ws(int64_t N, int64_t K, int group, bool pairs) {
  LinearWs w = {};
  if (!pairs) return w;
  w.lds = round_up(N, 4);
  w.scales = align256(static_cast<size_t>(N) * static_cast<size_t>(K) * 2);
  w.total = align256(w.scales + static_cast<size_t>(w.lds) * static_cast<size_t>((K + group - 1) / group) * 4);
  return w;
}

struct MoeWs {
  size_t logits, h, part, powers, counters, total;
  int64_t ld_powers;
};
bool moe_sizes_ok(int64_t T, int64_t H, int64_t I, int64_t E, int topk) {
  return T >= 0 && T <= kW4MoeMaxT && H > 0 && I > 0 && H % 8 == 0 && I % 8 == 0 && H <= kW4MoeMaxDim && I <= kW4MoeMaxDim && E > 0 &&
         E <= kW4MoeMaxExperts && topk > 0 && topk <= kW4MoeMaxK && topk <= E && T * topk <= kW4MoeMaxEntries;
}
MoeWs moe_ws(int64_t T, int64_t H, int64_t I, int64_t E, int topk, bool shared) {
  MoeWs w;
  const size_t rows = static_cast<size_t>(T * (topk + (shared ? 1 : 0)));
  w.logits = 0;
  w.h = align256(static_cast<size_t>(T * E) * 4);
  w.part = align256(w.h + rows * static_cast<size_t>(I) * 2);
  // A slot's powers are done with when the first of its sums goes to `part`: they share its rows where a row holds a byte for each
  // panel of h.
  const int64_t panels = (I + 31) / 32;
  const size_t end = w.part + rows * static_cast<size_t>(H) * 4;
  const bool share = panels <= 4 * H;
  w.powers = share ? w.part : end;
  w.ld_powers = share ? 4 * H : panels;
  w.counters = align256(share ? end : end + rows * static_cast<size_t>(panels));
  w.total = align256(w.counters + (kW4MoeCounters + static_cast<size_t>((H + kW4PanelRows - 1) / kW4PanelRows)) * 4);
  return w;
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

size_t nvfp4_w4_prepared_bytes(int64_t G, int64_t N, int64_t K, int group, int has_zeros, int gated) {
  if (G <= 0 || N <= 0 || K <= 0 || K % 8 || G >= kMaxDim || !dims_ok(N, K) || (gated && N % 2) ||
      (group != 32 && group != 64 && group != 128) || G * w4_panels(N, gated != 0) * w4_blocks(K) > INT32_MAX)
    return 0;
  return static_cast<size_t>(prepared_bytes(G, N, K, group, has_zeros != 0, gated != 0));
}

nvfp4_status nvfp4_w4_prepare(const uint8_t *codes, const void *scales, const uint8_t *zeros, int dtype, int64_t G,
                              int64_t N, int64_t K, int group, int gated, uint8_t *out, void *stream) {
  NV_REQUIRE(G > 0 && N > 0 && K > 0, NVFP4_ERR_INVALID_ARG, "G=%lld N=%lld K=%lld", (long long)G, (long long)N, (long long)K);
  nvfp4_status st = check_w4(__func__, dtype, K, group);
  if (st != NVFP4_OK) return st;
  NV_REQUIRE(!gated || N % 2 == 0, NVFP4_ERR_UNSUPPORTED_SHAPE, "N=%lld rows do not split into gate and up", (long long)N);
  NV_REQUIRE(codes && scales && out, NVFP4_ERR_INVALID_ARG, "NULL pointer argument");
  const size_t bytes = nvfp4_w4_prepared_bytes(G, N, K, group, zeros != nullptr, gated);
  NV_REQUIRE(bytes > 0, NVFP4_ERR_UNSUPPORTED_SHAPE, "sizes too large: %lld x %lld x %lld", (long long)G, (long long)N, (long long)K);
  NV_REQUIRE(aligned(codes, 4) && aligned(scales, 2) && aligned(out, 16), NVFP4_ERR_MISALIGNED,
             "codes must be 4-byte and out 16-byte aligned");
  const int64_t n_groups = (K + group - 1) / group;
  st = check_disjoint(__func__, {flat(out, static_cast<int64_t>(bytes), 1)},
                      {flat(codes, G * N * (K / 2), 1), flat(scales, G * N * n_groups, 2), flat(zeros, G * N * n_groups, 1)});
  if (st != NVFP4_OK) return st;
  DeviceInfo *d;
  if ((st = device_info(__func__, &d)) != NVFP4_OK) return st;
  NV_CUDA(launch_w4_prepare(codes, static_cast<const uint16_t *>(scales), zeros, G, N, K, group, gated != 0, out,
                            static_cast<cudaStream_t>(stream)),
          "4-bit weight preparation launch");
  return NVFP4_OK;
}

size_t nvfp4_w4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int group) {
  if (M < 0 || N <= 0 || K <= 0 || K % 8 || !dims_ok(M, K) || !dims_ok(N, K) || !dims_ok(M, N) || (group != 32 && group != 64 && group != 128))
    return 0;
  return linear_ws(N, K, group, may_take_pairs(M, N, K, group)).total;
}

nvfp4_status nvfp4_w4_linear(const void *x, int dtype, int64_t M, int64_t K, int64_t ldx, int64_t N, const uint8_t *w,
                             int group, int has_zeros, void *y, void *ws, size_t ws_bytes, void *stream) {
  NV_REQUIRE(M >= 0 && K > 0 && N > 0, NVFP4_ERR_INVALID_ARG, "M=%lld K=%lld N=%lld", (long long)M, (long long)K, (long long)N);
  nvfp4_status st = check_w4(__func__, dtype, K, group);
  if (st != NVFP4_OK) return st;
  NV_REQUIRE(dims_ok(M, K) && dims_ok(N, K) && dims_ok(M, N) && w4_panels(N, false) * w4_blocks(K) <= INT32_MAX,
             NVFP4_ERR_UNSUPPORTED_SHAPE, "sizes too large: M=%lld K=%lld N=%lld", (long long)M, (long long)K, (long long)N);
  NV_REQUIRE(w && (y || M == 0), NVFP4_ERR_INVALID_ARG, "NULL pointer argument");
  if ((st = check_rows(__func__, x, M, K, ldx)) != NVFP4_OK) return st;
  NV_REQUIRE(aligned(w, 16) && aligned(y, 16), NVFP4_ERR_MISALIGNED, "w and y must be 16-byte aligned");
  const bool zeros = has_zeros != 0;
  const LinearWs L = linear_ws(N, K, group, takes_pairs(M, N, K, group));
  if ((st = check_ws(__func__, ws, ws_bytes, L.total)) != NVFP4_OK) return st;
  st = check_disjoint(__func__, {{y, M, N, N, 2}, flat(ws, static_cast<int64_t>(L.total), 1)},
                      {{x, M, ldx, K, 2}, flat(w, prepared_bytes(1, N, K, group, zeros, false), 1)});
  if (st != NVFP4_OK) return st;
  DeviceInfo *d;
  if ((st = device_info(__func__, &d)) != NVFP4_OK) return st;
  if (M == 0) return NVFP4_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  W4Args a = {};
  a.x = x;
  a.ldx = ldx;
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.K = static_cast<int>(K);
  a.w = w;
  a.y = y;
  a.err = d->flags;
  if (M <= kStreamMaxTokens) {
    const int tok8 = M <= 8 ? 1 : 2, blocks = static_cast<int>(w4_blocks(K));
    const int splits = stream_splits(w4_panels(N, false), blocks, d->sms);
    const int rank = (blocks + splits - 1) / splits;
    int depth = (rank + 7) / 8;
    const int fit = (233472 / 2 - 2048) / (8 * w4_block_bytes(kW4BlockK / group, zeros));
    if (depth > fit) depth = fit;
    if (depth > 4) depth = 4;
    if (depth < tok8) depth = tok8;  // the ring holds a warp's sums at the end
    NV_CUDA(launch_w4_stream(a, dtype, group, zeros, tok8, splits, depth, s), "4-bit linear launch");
    return NVFP4_OK;
  }
  if (L.total == 0) {
    const TcPlan p = tc_plan(M, N, K, group);
    CUtensorMap mx;
    if ((st = make_map(__func__, &mx, x, K * 2, M, ldx * 2, p.tok)) != NVFP4_OK) return st;
    NV_CUDA(launch_w4_tc(mx, a, dtype, group, zeros, p.tok, p.splits, s), "4-bit linear launch");
    return NVFP4_OK;
  }
  uint16_t *ints = static_cast<uint16_t *>(ws);
  float *scales = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + L.scales);
  const int cols = pair_plan(M, N, K, group).cols;
  CUtensorMap mw, mx, my = {};
  if ((st = make_map(__func__, &mw, ints, K * 2, N, K * 2, kTHalf)) != NVFP4_OK) return st;
  if ((st = make_map(__func__, &mx, x, K * 2, M, ldx * 2, cols / 2)) != NVFP4_OK) return st;
  if (N % 8 == 0 && (st = make_map(__func__, &my, y, N * 2, M, N * 2, 32, 64, CU_TENSOR_MAP_SWIZZLE_NONE)) != NVFP4_OK) return st;
  TileArgs t = {};
  t.M = a.N;
  t.N = a.M;
  t.k_blocks = static_cast<int>((K + 63) / 64);
  t.groups = static_cast<int>((K + group - 1) / group);
  t.sa = scales;
  t.ld_sa = L.lds;
  t.out = y;
  t.ldo = N;
  t.err = d->flags;
  NV_CUDA(launch_w4_expand(a, dtype, group, zeros, ints, scales, L.lds, s), "4-bit weight expansion launch");
  NV_CUDA(in_pair_turn(d, s, [&] { return launch_w4_tile_gemm(mw, mx, my, t, dtype, group, cols, s); }), "4-bit tile GEMM launch");
  return NVFP4_OK;
}

size_t nvfp4_w4_moe_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t E, int topk, int has_shared) {
  return moe_sizes_ok(T, H, I, E, topk) ? moe_ws(T, H, I, E, topk, has_shared != 0).total : 0;
}

nvfp4_status nvfp4_w4_moe(const void *x, int dtype, int64_t T, int64_t H, int64_t ldx, int64_t I, int64_t E, int topk,
                          const void *router, const uint8_t *w13, const uint8_t *w2, const uint8_t *sh_w13,
                          const uint8_t *sh_w2, int group, int has_zeros, int act, void *y, void *ws, size_t ws_bytes,
                          void *stream) {
  NV_REQUIRE(T >= 0 && H > 0 && I > 0 && E > 0 && topk > 0, NVFP4_ERR_INVALID_ARG, "T=%lld H=%lld I=%lld E=%lld topk=%d",
             (long long)T, (long long)H, (long long)I, (long long)E, topk);
  nvfp4_status st = check_w4(__func__, dtype, H, group);
  if (st != NVFP4_OK) return st;
  NV_REQUIRE(act == NVFP4_ACT_SILU || act == NVFP4_ACT_GELU || act == NVFP4_ACT_GELU_TANH, NVFP4_ERR_INVALID_ARG, "activation %d", act);
  NV_REQUIRE(moe_sizes_ok(T, H, I, E, topk), NVFP4_ERR_UNSUPPORTED_SHAPE,
             "T=%lld (at most %d, T topk at most %d), H=%lld and I=%lld (multiples of 8, at most %lld), E=%lld (at most %lld), "
             "topk=%d (at most %d and E)",
             (long long)T, kW4MoeMaxT, kW4MoeMaxEntries, (long long)H, (long long)I, (long long)kW4MoeMaxDim, (long long)E,
             (long long)kW4MoeMaxExperts, topk, kW4MoeMaxK);
  NV_REQUIRE(router && w13 && w2 && (y || T == 0), NVFP4_ERR_INVALID_ARG, "NULL pointer argument");
  NV_REQUIRE((sh_w13 == nullptr) == (sh_w2 == nullptr), NVFP4_ERR_INVALID_ARG, "the shared expert's weights come together");
  if ((st = check_rows(__func__, x, T, H, ldx)) != NVFP4_OK) return st;
  NV_REQUIRE(aligned(router, 16) && aligned(w13, 16) && aligned(w2, 16) && aligned(sh_w13, 16) && aligned(sh_w2, 16) && aligned(y, 16),
             NVFP4_ERR_MISALIGNED, "router, weights and y must be 16-byte aligned");
  const bool zeros = has_zeros != 0, shared = sh_w13 != nullptr;
  const MoeWs L = moe_ws(T, H, I, E, topk, shared);
  if ((st = check_ws(__func__, ws, ws_bytes, L.total)) != NVFP4_OK) return st;
  st = check_disjoint(__func__, {flat(y, T * H, 2), flat(ws, static_cast<int64_t>(L.total), 1)},
                      {{x, T, ldx, H, 2}, flat(router, E * H, 2), flat(w13, prepared_bytes(E, 2 * I, H, group, zeros, true), 1),
                       flat(w2, prepared_bytes(E, H, I, group, zeros, false), 1),
                       flat(sh_w13, prepared_bytes(1, 2 * I, H, group, zeros, true), 1),
                       flat(sh_w2, prepared_bytes(1, H, I, group, zeros, false), 1)});
  if (st != NVFP4_OK) return st;
  DeviceInfo *d;
  if ((st = device_info(__func__, &d)) != NVFP4_OK) return st;
  if (T == 0) return NVFP4_OK;
  uint8_t *p = static_cast<uint8_t *>(ws);
  W4MoeArgs a = {};
  a.x = x;
  a.ldx = ldx;
  a.T = static_cast<int>(T);
  a.H = static_cast<int>(H);
  a.I = static_cast<int>(I);
  a.E = static_cast<int>(E);
  a.topk = topk;
  a.router = router;
  a.w13 = w13;
  a.w2 = w2;
  a.sh13 = sh_w13;
  a.sh2 = sh_w2;
  a.act = act;
  a.y = y;
  a.logits = reinterpret_cast<float *>(p + L.logits);
  a.h = reinterpret_cast<uint16_t *>(p + L.h);
  a.part = reinterpret_cast<float *>(p + L.part);
  a.powers = p + L.powers;
  a.ld_powers = L.ld_powers;
  a.counters = reinterpret_cast<int *>(p + L.counters);
  a.err = d->flags;
  NV_CUDA(launch_w4_moe(a, dtype, group, zeros, d->sms, static_cast<cudaStream_t>(stream)), "4-bit mixture-of-experts launch");
  return NVFP4_OK;
}

}  // extern "C"
