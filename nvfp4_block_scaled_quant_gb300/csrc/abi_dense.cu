// Host side of the dense feed-forward operators' C ABI: argument validation, the choice between
// the weight-streaming and the tile GEMM, tensor maps, workspace layout and launch sequences.
#include <cstring>
#include <initializer_list>

#include "abi_util.h"
#include "dense.h"
#include "stream_gemm.cuh"
#include "tile_gemm.cuh"

namespace nvfp4 {
namespace {

constexpr int64_t kMaxDim = int64_t(1) << 24;
constexpr int64_t kMaxArea = int64_t(1) << 40;

bool dtype16(int d) { return d == NVFP4_DT_BF16 || d == NVFP4_DT_FP16; }
bool dims_ok(int64_t a, int64_t b) { return a < kMaxDim && b < kMaxDim && a * b < kMaxArea; }

#define NV_DIMS(a, b)                                                                                \
  NV_REQUIRE(dims_ok(a, b), NVFP4_ERR_UNSUPPORTED_SHAPE, "sizes too large: %lld x %lld", (long long)(a), \
             (long long)(b))

// `rows` rows of `cols` elements of `bytes` bytes, `ld` elements apart, taken as the whole range from the first
// element to the last.
struct Span {
  const void *p;
  int64_t rows, ld, cols, bytes;
};
bool overlap(const Span &a, const Span &b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.cols <= 0 || b.cols <= 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  const uintptr_t a1 = a0 + static_cast<uintptr_t>(((a.rows - 1) * a.ld + a.cols) * a.bytes);
  const uintptr_t b1 = b0 + static_cast<uintptr_t>(((b.rows - 1) * b.ld + b.cols) * b.bytes);
  return a0 < b1 && b0 < a1;
}
Span flat(const void *p, int64_t n, int64_t bytes) { return {p, 1, n, n, bytes}; }

// Refuses what is written (outputs, the workspace) inside what is read, which other blocks may still be
// reading, and inside what else is written.
nvfp4_status check_disjoint(const char *fn, std::initializer_list<Span> written, std::initializer_list<Span> read) {
  for (auto w = written.begin(); w != written.end(); ++w) {
    for (const Span &r : read)
      if (overlap(*w, r)) return fail(NVFP4_ERR_INVALID_ARG, fn, "an output or the workspace overlaps an input");
    for (auto o = written.begin(); o != w; ++o)
      if (overlap(*w, *o)) return fail(NVFP4_ERR_INVALID_ARG, fn, "outputs and workspace overlap one another");
  }
  return NVFP4_OK;
}

// Estimated times (in units of 10 ns) that choose between the GEMMs.  The coefficients were fitted to
// times on a GB300 over M = 16 .. 2048 and five (K, N) between 512 x 512 and 7168 x 7168; they rank
// the choices, nothing else depends on them.
struct Cost {
  int64_t start;             // of a launch
  int64_t block256, block128;  // a K block of a 256- or 128-column pair tile
  int64_t tile;              // a tile's start and end
  int64_t tok_start[4], tok_block[4];  // weight-streaming GEMM of 16, 32, 64, 128 tokens
};
constexpr Cost kFp8Cost = {200, 46, 32, 160, {220, 250, 350, 500}, {40, 45, 60, 110}};
constexpr Cost kGatedCost = {250, 33, 24, 200, {220, 250, 330, 0}, {50, 65, 78, 0}};

// How the weight-streaming GEMM covers M tokens and N features: token tiles of `tok` columns and
// clusters of `splits` CTAs along K.  A choice costs its waves of CTAs (two per SM) times a CTA's K
// blocks plus a fixed part (start-up, reduction) of about four.
struct StreamPlan {
  int tok, splits;
  int64_t cost;
};
StreamPlan stream_plan(int64_t M, int64_t N, int k_blocks, int max_tok, int sms, const Cost &c) {
  StreamPlan p = {16, 0, 0};
  int size = 0;
  while (p.tok < max_tok && p.tok < M) p.tok *= 2, ++size;
  const int64_t tiles = ((N + 127) / 128) * ((M + p.tok - 1) / p.tok);
  int64_t best = 0;
  for (int s = 1; s <= kStreamMaxSplit && s <= k_blocks; ++s) {
    const int64_t waves = (tiles * s + 2 * sms - 1) / (2 * sms);
    const int64_t blocks = waves * ((k_blocks + s - 1) / s + 4);
    if (p.splits == 0 || blocks < best) {
      best = blocks;
      p.splits = s;
    }
  }
  p.cost = c.tok_start[size] + best * c.tok_block[size];
  return p;
}

// Accumulator columns of the pair tiles for M x N outputs: 256, or 128 where the waves of tiles (one
// pair per two SMs) then take less time.  out_cols: output columns of a 256-column tile.
struct TilePlan {
  int cols;
  int64_t cost;
};
TilePlan tile_plan(int64_t M, int64_t N, int k_blocks, int out_cols, int sms, const Cost &c) {
  const int64_t m = (M + kTRows - 1) / kTRows, pairs = sms / 2;
  const int64_t w = m * ((N + out_cols - 1) / out_cols), n = m * ((N + out_cols / 2 - 1) / (out_cols / 2));
  const int64_t cost_w = (w + pairs - 1) / pairs * (k_blocks * c.block256 + c.tile);
  const int64_t cost_n = (n + pairs - 1) / pairs * (k_blocks * c.block128 + c.tile);
  return cost_n < cost_w ? TilePlan{128, c.start + cost_n} : TilePlan{256, c.start + cost_w};
}

// The two products of the gradients in one launch: columns of the tiles, and how many rounds of dW's tiles
// the pairs take that have one tile of dx less than the others (TileOp::kGrad), from the longest pair's time.
struct GradPlan {
  int cols, early;
};
GradPlan grad_plan(int64_t M, int64_t dw_M, int64_t N, int k_blocks, int dw_k_blocks, int sms, const Cost &c) {
  GradPlan best = {256, 0};
  int64_t best_time = -1;
  for (int cols = 256; cols >= 128; cols /= 2) {
    const int64_t n = (N + cols - 1) / cols, block = cols == 256 ? c.block256 : c.block128;
    const int64_t total = (M + kTRows - 1) / kTRows * n, dw_total = (dw_M + kTRows - 1) / kTRows * n;
    const int64_t time = k_blocks * block + c.tile, dw_time = dw_k_blocks * block + c.tile;
    const int64_t pairs = total + dw_total < sms / 2 ? total + dw_total : sms / 2;
    const int64_t behind = total % pairs, rest = pairs - behind;
    const int64_t fit = behind ? time / dw_time : 0;  // tiles of dW in the time of one of dx
    for (int64_t early = fit; early <= (behind ? fit + 1 : 0); ++early) {
      const int64_t base = dw_total < early * rest ? dw_total : early * rest, left = dw_total - base;
      // the first pair with and the first without a tile in dx's last round (the others take no longer)
      const int64_t with = (total / pairs + 1) * time + (left > rest ? (left - 1 - rest) / pairs + 1 : 0) * dw_time;
      const int64_t without = total / pairs * time + ((base + rest - 1) / rest + (left + pairs - 1) / pairs) * dw_time;
      const int64_t longest = behind && with > without ? with : without;
      if (best_time < 0 || longest < best_time) {
        best_time = longest;
        best = {cols, static_cast<int>(early)};
      }
    }
  }
  return best;
}

// The weight-streaming GEMM is considered up to kStreamMaxM rows (its token tiles re-read the weights),
// and taken up to kStreamMinM whatever the estimates: a pair tile's 128-row boxes of a tensor of 64
// rows or fewer load at half speed (1536 -> 16384: 22 us for M = 64, 10.5 us for M = 100).
constexpr int64_t kStreamMinM = 64;
constexpr int64_t kStreamMaxM = 256;
constexpr int kFp8StreamTok = 128;
constexpr int kGatedStreamTok = 64;

nvfp4_status fp8_gemm_impl(const char *fn, DeviceInfo *d, const uint8_t *xq, const float *xs, int64_t lds, int64_t M,
                           int64_t K, int64_t N, const uint8_t *w, const float *w_s, int dtype, void *y,
                           cudaStream_t s) {
  const int k_blocks = static_cast<int>((K + 127) / 128);
  CUtensorMap mx, mw;
  nvfp4_status st;
  const TilePlan tp = tile_plan(M, N, k_blocks, 256, d->sms, kFp8Cost);
  const StreamPlan p = stream_plan(M, N, k_blocks, kFp8StreamTok, d->sms, kFp8Cost);
  if (M <= kStreamMinM || (M <= kStreamMaxM && p.cost <= tp.cost)) {
    if ((st = make_map(fn, &mx, xq, K, M, K, p.tok)) != NVFP4_OK) return st;
    if ((st = make_map(fn, &mw, w, K, N, K, 128)) != NVFP4_OK) return st;
    StreamArgs a = {};
    a.M = static_cast<int>(M);
    a.N = static_cast<int>(N);
    a.k_blocks = k_blocks;
    a.sa = xs;
    a.ld_sa = lds;
    a.sw = w_s;
    a.out = y;
    a.ldo = N;
    a.err = d->flags;
    NV_CUDA(launch_fp8_stream_gemm(mw, mx, a, dtype, p.tok, p.splits, s), "FP8 streaming GEMM launch");
    return NVFP4_OK;
  }
  if ((st = make_map(fn, &mx, xq, K, M, K, kTHalf)) != NVFP4_OK) return st;
  if ((st = make_map(fn, &mw, w, K, N, K, tp.cols / 2)) != NVFP4_OK) return st;
  TileArgs a = {};
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.k_blocks = k_blocks;
  a.sa = xs;
  a.ld_sa = lds;
  a.sw = w_s;
  a.out = y;
  a.ldo = N;
  a.err = d->flags;
  NV_CUDA(in_pair_turn(d, s, [&] { return launch_fp8_tile_gemm(mx, mw, a, dtype, tp.cols, s); }), "FP8 tile GEMM launch");
  return NVFP4_OK;
}

nvfp4_status check_fp8_x(const char *fn, const void *x, int dtype, int64_t M, int64_t K, int64_t ldx) {
  if (!(M >= 0 && K > 0)) return fail(NVFP4_ERR_INVALID_ARG, fn, "M=%lld K=%lld", (long long)M, (long long)K);
  if (!dtype16(dtype)) return fail(NVFP4_ERR_INVALID_ARG, fn, "dtype %d is neither bf16 nor fp16", dtype);
  if (K % 16) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, fn, "K=%lld must be a multiple of 16", (long long)K);
  if (!dims_ok(M, K)) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, fn, "sizes too large");
  if (!x && M > 0) return fail(NVFP4_ERR_INVALID_ARG, fn, "x is NULL");
  if (ldx < K || ldx % 8 || ldx >= kMaxDim * 16)
    return fail(NVFP4_ERR_MISALIGNED, fn, "row stride %lld must be >= %lld and a multiple of 8", (long long)ldx,
                (long long)K);
  if (!aligned(x, 16)) return fail(NVFP4_ERR_MISALIGNED, fn, "x must be 16-byte aligned");
  return NVFP4_OK;
}

// Whether the weight-streaming GEMM quantises the activations itself.  That saves a launch (about 3 us
// of GPU time, and of the host's), but every CTA encodes the rows of its K blocks again: it pays up to
// one token tile of 16 rows, and up to 64 rows while the product is small.  GPU time in one launch / two:
// 7168 -> 7168 of 1 row 9.1 / 13.3 us, of 8 rows 10.9 / 11.7, of 16 rows 14.9 / 13.2 (the host's time
// still favours one), of 32 rows 24 / 14; 2000 -> 1136 of 24 rows 7.6 / 7.5, of 64 rows 8.2 / 8.8;
// 512 x 512 of 24 rows 6.5 / 7.8, of 64 rows 6.6 / 9.0; 2048 -> 7168 of 32 rows 12.1 / 9.7.
constexpr int64_t kFp8FusedM = 16, kFp8FusedSmallM = 64, kFp8FusedSmallMnk = int64_t(1) << 27;
constexpr int kFp8FusedTok = 32;
bool quantise_in_gemm(int64_t M, int64_t K, int64_t N) {
  return M <= kFp8FusedM || (M <= kFp8FusedSmallM && M * N * K <= kFp8FusedSmallMnk);
}

struct Fp8Ws {
  size_t q, s, total;
  int64_t lds;
};
Fp8Ws fp8_ws(int64_t M, int64_t K) {
  Fp8Ws w = {};
  if (M <= kFp8FusedM) return w;  // quantised in the GEMM
  w.lds = round_up(M, 4);
  w.q = 0;
  w.s = align256(static_cast<size_t>(M) * static_cast<size_t>(K));
  w.total = align256(w.s + static_cast<size_t>(w.lds) * static_cast<size_t>((K + 127) / 128) * 4);
  return w;
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

// ---------------------------------------------------------------- FP8 block-scaled linear

nvfp4_status nvfp4_fp8_quantize_act(const void *x, int dtype, int64_t M, int64_t K, int64_t ldx, uint8_t *q, float *xs,
                                    int64_t lds, void *stream) {
  nvfp4_status st = check_fp8_x(__func__, x, dtype, M, K, ldx);
  if (st != NVFP4_OK) return st;
  NV_REQUIRE((q && xs) || M == 0, NVFP4_ERR_INVALID_ARG, "NULL pointer argument");
  NV_REQUIRE(lds >= M && lds % 4 == 0 && lds < kMaxDim * 16, NVFP4_ERR_MISALIGNED,
             "lds=%lld must be >= M and a multiple of 4", (long long)lds);
  NV_REQUIRE(aligned(q, 16) && aligned(xs, 16), NVFP4_ERR_MISALIGNED, "q and xs must be 16-byte aligned");
  DeviceInfo *d;
  if ((st = device_info(__func__, &d)) != NVFP4_OK) return st;
  st = check_disjoint(__func__, {{q, M, K, K, 1}, {xs, (K + 127) / 128, lds, M, 4}}, {{x, M, ldx, K, 2}});
  if (st != NVFP4_OK) return st;
  if (M == 0) return NVFP4_OK;
  NV_CUDA(launch_fp8_quantize_act(x, dtype, M, K, ldx, q, xs, lds, d->sms, static_cast<cudaStream_t>(stream)),
          "FP8 quantise launch");
  return NVFP4_OK;
}

nvfp4_status nvfp4_fp8_quantize_weight(const void *w, int dtype, int64_t N, int64_t K, int64_t ldw, uint8_t *q,
                                       float *w_s, void *stream) {
  nvfp4_status st = check_fp8_x(__func__, w, dtype, N, K, ldw);
  if (st != NVFP4_OK) return st;
  NV_REQUIRE(N > 0, NVFP4_ERR_INVALID_ARG, "N=%lld", (long long)N);
  NV_REQUIRE(N <= 65535 * 128, NVFP4_ERR_UNSUPPORTED_SHAPE, "N=%lld too large", (long long)N);
  NV_REQUIRE(q && w_s, NVFP4_ERR_INVALID_ARG, "NULL pointer argument");
  NV_REQUIRE(aligned(q, 16) && aligned(w_s, 4), NVFP4_ERR_MISALIGNED, "q must be 16-byte aligned");
  st = check_disjoint(__func__, {{q, N, K, K, 1}, flat(w_s, (N + 127) / 128 * ((K + 127) / 128), 4)}, {{w, N, ldw, K, 2}});
  if (st != NVFP4_OK) return st;
  DeviceInfo *d;
  if ((st = device_info(__func__, &d)) != NVFP4_OK) return st;
  NV_CUDA(launch_fp8_quantize_weight(w, dtype, N, K, ldw, q, w_s, static_cast<cudaStream_t>(stream)),
          "FP8 weight quantise launch");
  return NVFP4_OK;
}

nvfp4_status nvfp4_fp8_gemm(const uint8_t *xq, const float *xs, int64_t lds, int64_t M, int64_t K, int64_t N,
                            const uint8_t *w, const float *w_s, int dtype, void *y, void *stream) {
  NV_REQUIRE(M >= 0 && K > 0 && N > 0, NVFP4_ERR_INVALID_ARG, "M=%lld K=%lld N=%lld", (long long)M, (long long)K,
             (long long)N);
  NV_REQUIRE(dtype16(dtype), NVFP4_ERR_INVALID_ARG, "dtype %d is neither bf16 nor fp16", dtype);
  NV_REQUIRE(K % 16 == 0, NVFP4_ERR_UNSUPPORTED_SHAPE, "K=%lld must be a multiple of 16", (long long)K);
  NV_DIMS(M, K);
  NV_DIMS(N, K);
  NV_DIMS(M, N);
  NV_REQUIRE((xq && xs && y) || M == 0, NVFP4_ERR_INVALID_ARG, "NULL pointer argument");
  NV_REQUIRE(w && w_s, NVFP4_ERR_INVALID_ARG, "NULL pointer argument");
  NV_REQUIRE(lds >= M && lds % 4 == 0 && lds < kMaxDim * 16, NVFP4_ERR_MISALIGNED,
             "lds=%lld must be >= M and a multiple of 4", (long long)lds);
  NV_REQUIRE(aligned(xq, 16) && aligned(xs, 16) && aligned(w, 16) && aligned(w_s, 4) && aligned(y, 16),
             NVFP4_ERR_MISALIGNED, "xq, xs, w and y must be 16-byte aligned");
  const int64_t k_blocks = (K + 127) / 128;
  nvfp4_status st = check_disjoint(__func__, {{y, M, N, N, 2}},
                                   {{xq, M, K, K, 1}, {xs, k_blocks, lds, M, 4}, flat(w, N * K, 1),
                                    flat(w_s, (N + 127) / 128 * k_blocks, 4)});
  if (st != NVFP4_OK) return st;
  DeviceInfo *d;
  if ((st = device_info(__func__, &d)) != NVFP4_OK) return st;
  if (M == 0) return NVFP4_OK;
  return fp8_gemm_impl(__func__, d, xq, xs, lds, M, K, N, w, w_s, dtype, y, static_cast<cudaStream_t>(stream));
}

size_t nvfp4_fp8_linear_workspace_bytes(int64_t M, int64_t K) {
  if (M < 0 || K <= 0 || K % 16 || !dims_ok(M, K)) return 0;
  return fp8_ws(M, K).total;
}

nvfp4_status nvfp4_fp8_linear(const void *x, int dtype, int64_t M, int64_t K, int64_t ldx, int64_t N, const uint8_t *w,
                              const float *w_s, void *y, void *ws, size_t ws_bytes, void *stream) {
  nvfp4_status st = check_fp8_x(__func__, x, dtype, M, K, ldx);
  if (st != NVFP4_OK) return st;
  NV_REQUIRE(N > 0, NVFP4_ERR_INVALID_ARG, "N=%lld", (long long)N);
  NV_DIMS(N, K);
  NV_DIMS(M, N);
  NV_REQUIRE(w && w_s && (y || M == 0), NVFP4_ERR_INVALID_ARG, "NULL pointer argument");
  NV_REQUIRE(aligned(w, 16) && aligned(w_s, 4) && aligned(y, 16), NVFP4_ERR_MISALIGNED,
             "w and y must be 16-byte aligned");
  const Fp8Ws L = fp8_ws(M, K);
  if ((st = check_ws(__func__, ws, ws_bytes, L.total)) != NVFP4_OK) return st;
  st = check_disjoint(__func__, {{y, M, N, N, 2}, flat(ws, static_cast<int64_t>(L.total), 1)},
                      {{x, M, ldx, K, 2}, flat(w, N * K, 1), flat(w_s, (N + 127) / 128 * ((K + 127) / 128), 4)});
  if (st != NVFP4_OK) return st;
  DeviceInfo *d;
  if ((st = device_info(__func__, &d)) != NVFP4_OK) return st;
  if (M == 0) return NVFP4_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (quantise_in_gemm(M, K, N)) {
    CUtensorMap mw;
    if ((st = make_map(__func__, &mw, w, K, N, K, 128)) != NVFP4_OK) return st;
    StreamArgs a = {};
    a.M = static_cast<int>(M);
    a.N = static_cast<int>(N);
    a.K = static_cast<int>(K);
    a.k_blocks = static_cast<int>((K + 127) / 128);
    a.sw = w_s;
    a.out = y;
    a.ldo = N;
    a.x = x;
    a.ldx = ldx;
    a.err = d->flags;
    // the splits of the product after a quantiser: the same sums in the same order
    const StreamPlan p = stream_plan(M, N, a.k_blocks, kFp8StreamTok, d->sms, kFp8Cost);
    NV_CUDA(launch_fp8_stream_linear(mw, a, dtype, p.tok < kFp8FusedTok ? p.tok : kFp8FusedTok, p.splits, s),
            "FP8 linear launch");
    return NVFP4_OK;
  }
  uint8_t *q = static_cast<uint8_t *>(ws) + L.q;
  float *xs = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + L.s);
  NV_CUDA(launch_fp8_quantize_act(x, dtype, M, K, ldx, q, xs, L.lds, d->sms, s), "FP8 quantise launch");
  return fp8_gemm_impl(__func__, d, q, xs, L.lds, M, K, N, w, w_s, dtype, y, s);
}

// ---------------------------------------------------------------- gated linear

static nvfp4_status check_gated(const char *fn, const void *x, int dtype, int64_t T, int64_t H, int64_t ldx, int64_t I,
                                const void *wg, const void *wu, int act) {
  if (!(T >= 0 && H > 0 && I > 0))
    return fail(NVFP4_ERR_INVALID_ARG, fn, "T=%lld H=%lld I=%lld", (long long)T, (long long)H, (long long)I);
  if (!dtype16(dtype)) return fail(NVFP4_ERR_INVALID_ARG, fn, "dtype %d is neither bf16 nor fp16", dtype);
  if (act != NVFP4_ACT_SILU && act != NVFP4_ACT_GELU && act != NVFP4_ACT_GELU_TANH)
    return fail(NVFP4_ERR_INVALID_ARG, fn, "activation %d", act);
  if (H % 8 || I % 8)
    return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, fn, "H=%lld and I=%lld must be multiples of 8", (long long)H, (long long)I);
  if (!dims_ok(T, H) || !dims_ok(T, 2 * I) || !dims_ok(2 * I, H))
    return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, fn, "sizes too large");
  if (!wg || !wu || (!x && T > 0)) return fail(NVFP4_ERR_INVALID_ARG, fn, "NULL pointer argument");
  if (ldx < H || ldx % 8 || ldx >= kMaxDim * 16)
    return fail(NVFP4_ERR_MISALIGNED, fn, "row stride %lld must be >= %lld and a multiple of 8", (long long)ldx,
                (long long)H);
  if (!aligned(x, 16) || !aligned(wg, 16) || !aligned(wu, 16))
    return fail(NVFP4_ERR_MISALIGNED, fn, "x, w_gate and w_up must be 16-byte aligned");
  return NVFP4_OK;
}

nvfp4_status nvfp4_gated_linear(const void *x, int dtype, int64_t T, int64_t H, int64_t ldx, int64_t I,
                                const void *w_gate, const void *w_up, int act, void *h, float *gu, void *stream) {
  nvfp4_status st = check_gated(__func__, x, dtype, T, H, ldx, I, w_gate, w_up, act);
  if (st != NVFP4_OK) return st;
  NV_REQUIRE(h || T == 0, NVFP4_ERR_INVALID_ARG, "h is NULL");
  NV_REQUIRE(aligned(h, 16) && aligned(gu, 32), NVFP4_ERR_MISALIGNED, "h must be 16-byte and gu 32-byte aligned");
  st = check_disjoint(__func__, {{h, T, I, I, 2}, flat(gu, 2 * T * I, 4)},
                      {{x, T, ldx, H, 2}, flat(w_gate, I * H, 2), flat(w_up, I * H, 2)});
  if (st != NVFP4_OK) return st;
  DeviceInfo *d;
  if ((st = device_info(__func__, &d)) != NVFP4_OK) return st;
  if (T == 0) return NVFP4_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int k_blocks = static_cast<int>((H + 63) / 64);
  CUtensorMap mx, mg, mu;
  const TilePlan tp = tile_plan(T, I, k_blocks, 128, d->sms, kGatedCost);
  const StreamPlan p = stream_plan(T, I, k_blocks, kGatedStreamTok, d->sms, kGatedCost);
  const bool stream_weights = T <= kStreamMinM || (T <= kStreamMaxM && p.cost <= tp.cost);
  const int cols = stream_weights ? 256 : tp.cols;
  if ((st = make_map(__func__, &mg, w_gate, H * 2, I, H * 2, cols / 2)) != NVFP4_OK) return st;
  if ((st = make_map(__func__, &mu, w_up, H * 2, I, H * 2, cols / 2)) != NVFP4_OK) return st;
  if (stream_weights) {
    if ((st = make_map(__func__, &mx, x, H * 2, T, ldx * 2, p.tok)) != NVFP4_OK) return st;
    StreamArgs a = {};
    a.M = static_cast<int>(T);
    a.N = static_cast<int>(I);
    a.k_blocks = k_blocks;
    a.out = h;
    a.ldo = I;
    a.save = gu;
    a.err = d->flags;
    NV_CUDA(launch_gated_stream_gemm(mx, mg, mu, a, dtype, act, p.tok, p.splits, s), "gated streaming GEMM launch");
    return NVFP4_OK;
  }
  if ((st = make_map(__func__, &mx, x, H * 2, T, ldx * 2, kTHalf)) != NVFP4_OK) return st;
  TileArgs a = {};
  a.M = static_cast<int>(T);
  a.N = static_cast<int>(I);
  a.k_blocks = k_blocks;
  a.out = h;
  a.ldo = I;
  a.save = gu;
  a.err = d->flags;
  NV_CUDA(in_pair_turn(d, s, [&] { return launch_gated_tile_gemm(mx, mg, mu, a, dtype, act, cols, s); }),
          "gated tile GEMM launch");
  return NVFP4_OK;
}

size_t nvfp4_gated_linear_backward_workspace_bytes_dt(int64_t T, int64_t I, int dtype) {
  if (T < 0 || I <= 0 || I % 8 || !dims_ok(T, 2 * I) || !dtype16(dtype)) return 0;
  const size_t pair = align256(static_cast<size_t>(T) * static_cast<size_t>(I) * 4);
  return pair + (dtype == NVFP4_DT_FP16 && T > 0 ? align256((kGatedGradParts + 1) * 4) : 0);
}

size_t nvfp4_gated_linear_backward_workspace_bytes(int64_t T, int64_t I) {
  return nvfp4_gated_linear_backward_workspace_bytes_dt(T, I, NVFP4_DT_BF16);
}

nvfp4_status nvfp4_gated_linear_backward(const void *dh, int64_t lddh, const void *x, int64_t ldx, int dtype, int64_t T,
                                         int64_t H, int64_t I, const void *w_gate, const void *w_up, int act,
                                         const float *gu, void *dx, void *dw_gate, void *dw_up, void *ws,
                                         size_t ws_bytes, void *stream) {
  nvfp4_status st = check_gated(__func__, x, dtype, T, H, ldx, I, w_gate, w_up, act);
  if (st != NVFP4_OK) return st;
  NV_REQUIRE((dh && gu) || T == 0, NVFP4_ERR_INVALID_ARG, "NULL pointer argument");
  NV_REQUIRE((dw_gate == nullptr) == (dw_up == nullptr), NVFP4_ERR_INVALID_ARG, "dw_gate and dw_up come together");
  NV_REQUIRE(lddh >= I && lddh % 8 == 0 && lddh < kMaxDim * 16, NVFP4_ERR_MISALIGNED,
             "lddh=%lld must be >= I and a multiple of 8", (long long)lddh);
  NV_REQUIRE(aligned(dh, 16) && aligned(gu, 16) && aligned(dx, 16) && aligned(dw_gate, 16) && aligned(dw_up, 16),
             NVFP4_ERR_MISALIGNED, "pointers must be 16-byte aligned");
  const size_t need = nvfp4_gated_linear_backward_workspace_bytes_dt(T, I, dtype);
  if ((st = check_ws(__func__, ws, ws_bytes, need)) != NVFP4_OK) return st;
  st = check_disjoint(__func__,
                      {flat(dx, T * H, 2), flat(dw_gate, I * H, 2), flat(dw_up, I * H, 2), flat(ws, static_cast<int64_t>(need), 1)},
                      {{dh, T, lddh, I, 2}, {x, T, ldx, H, 2}, flat(w_gate, I * H, 2), flat(w_up, I * H, 2), flat(gu, 2 * T * I, 4)});
  if (st != NVFP4_OK) return st;
  DeviceInfo *d;
  if ((st = device_info(__func__, &d)) != NVFP4_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    if (dw_gate) {
      NV_CUDA(cudaMemsetAsync(dw_gate, 0, static_cast<size_t>(I) * H * 2, s), "zero dw_gate");
      NV_CUDA(cudaMemsetAsync(dw_up, 0, static_cast<size_t>(I) * H * 2, s), "zero dw_up");
    }
    return NVFP4_OK;
  }
  if (!dx && !dw_gate) return NVFP4_OK;
  uint16_t *dgu = static_cast<uint16_t *>(ws);
  // fp16: the parts of the maximum and, behind them, the factor of the products' sums
  uint32_t *parts = reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(ws) + nvfp4_gated_linear_backward_workspace_bytes(T, I));
  float *unscale = reinterpret_cast<float *>(parts + kGatedGradParts);
  NV_CUDA(launch_gated_grad(dh, lddh, gu, T, I, dtype, act, dgu, parts, unscale, d->sms, s), "gated gradient launch");
  // an absent product's maps are not used: any valid one stands in
  CUtensorMap mdg, mdu, mg, mu, ma, mx;
  TileArgs a = {};
  a.N = static_cast<int>(H);
  a.ldo = H;
  a.unscale = unscale;
  a.err = d->flags;
  if (dx) {
    if ((st = make_map(__func__, &mdg, dgu, I * 2, T, I * 4, kTHalf)) != NVFP4_OK) return st;
    if ((st = make_map(__func__, &mdu, dgu + I, I * 2, T, I * 4, kTHalf)) != NVFP4_OK) return st;
    if ((st = make_map(__func__, &mg, w_gate, H * 2, I, H * 2, 64)) != NVFP4_OK) return st;
    if ((st = make_map(__func__, &mu, w_up, H * 2, I, H * 2, 64)) != NVFP4_OK) return st;
    a.M = static_cast<int>(T);
    a.k_blocks = static_cast<int>((I + 63) / 64);
    a.out = dx;
  }
  if (dw_gate) {
    if ((st = make_map(__func__, &ma, dgu, I * 4, T, I * 4, 64)) != NVFP4_OK) return st;
    if ((st = make_map(__func__, &mx, x, H * 2, T, ldx * 2, 64)) != NVFP4_OK) return st;
    a.dw_M = static_cast<int>(2 * I);
    a.dw_k_blocks = static_cast<int>((T + 63) / 64);
    a.dwg = dw_gate;
    a.dwu = dw_up;
  }
  if (!dx) mdg = mdu = ma, mg = mu = mx;
  if (!dw_gate) ma = mdg, mx = mg;
  const GradPlan p = grad_plan(a.M, a.dw_M, H, 2 * a.k_blocks, a.dw_k_blocks, d->sms, kGatedCost);
  a.early = p.early;
  NV_CUDA(in_pair_turn(d, s, [&] { return launch_gated_grad_gemm(mdg, mdu, mg, mu, ma, mx, a, dtype, p.cols, s); }),
          "gradient products launch");
  return NVFP4_OK;
}

// ---------------------------------------------------------------- residual norm

static nvfp4_status check_norm(const char *fn, const void *f, int dtype, const void *r, int r_dtype, int64_t M,
                               int64_t K, int64_t ldf, int64_t ldr, const void *ga, const void *gate, int gate_kind,
                               int64_t groups, float scale, const void *gb) {
  if (!(M >= 0 && K > 0)) return fail(NVFP4_ERR_INVALID_ARG, fn, "M=%lld K=%lld", (long long)M, (long long)K);
  if (!dtype16(dtype) || (r_dtype != dtype && r_dtype != NVFP4_DT_FP32))
    return fail(NVFP4_ERR_INVALID_ARG, fn, "dtype %d (bf16 or fp16) with residual dtype %d (the same or fp32)", dtype,
                r_dtype);
  if (K % 8 || K > kNormMaxK)
    return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, fn, "K=%lld must be a multiple of 8, at most %lld", (long long)K,
                (long long)kNormMaxK);
  if (!dims_ok(M, K)) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, fn, "sizes too large");
  if ((!f || !r) && M > 0) return fail(NVFP4_ERR_INVALID_ARG, fn, "NULL pointer argument");
  if (ldf < K || ldf % 8 || ldr < K || ldr % 8 || ldf >= kMaxDim * 16 || ldr >= kMaxDim * 16)
    return fail(NVFP4_ERR_MISALIGNED, fn, "row strides %lld, %lld must be >= K and multiples of 8", (long long)ldf,
                (long long)ldr);
  if (gate_kind != NVFP4_GATE_NONE && gate_kind != NVFP4_GATE_CHANNEL && gate_kind != NVFP4_GATE_ROW)
    return fail(NVFP4_ERR_INVALID_ARG, fn, "gate kind %d", gate_kind);
  // a gate of no rows has no address
  if ((gate_kind == NVFP4_GATE_NONE) != (gate == nullptr) && !(gate_kind == NVFP4_GATE_ROW && M == 0))
    return fail(NVFP4_ERR_INVALID_ARG, fn, "a gate and its kind come together");
  if (gate_kind == NVFP4_GATE_CHANNEL) {
    if (groups <= 0 || M % groups)
      return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, fn, "M=%lld rows in %lld groups", (long long)M, (long long)groups);
  }
  if (!(scale - scale == 0.f)) return fail(NVFP4_ERR_INVALID_ARG, fn, "scale must be finite");
  if (!aligned(f, 16) || !aligned(r, 16) || !aligned(ga, 16) || !aligned(gb, 16) ||
      !aligned(gate, gate_kind == NVFP4_GATE_ROW ? 2 : 16))
    return fail(NVFP4_ERR_MISALIGNED, fn, "f, r, the gammas and a channel gate must be 16-byte aligned");
  return NVFP4_OK;
}

nvfp4_status nvfp4_residual_norm(const void *f, int dtype, const void *r, int r_dtype, int64_t M, int64_t K,
                                 int64_t ldf, int64_t ldr, const void *gamma_after, const void *gate, int gate_kind,
                                 int64_t gate_groups, float scale, const void *gamma_before, float eps, void *r_out,
                                 void *y, float *stats, void *stream) {
  nvfp4_status st = check_norm(__func__, f, dtype, r, r_dtype, M, K, ldf, ldr, gamma_after, gate, gate_kind,
                               gate_groups, scale, gamma_before);
  if (st != NVFP4_OK) return st;
  NV_REQUIRE(eps >= 0.f && eps < 1e30f, NVFP4_ERR_INVALID_ARG, "eps must be finite and >= 0");
  NV_REQUIRE(r_out || M == 0, NVFP4_ERR_INVALID_ARG, "r_out is NULL");
  NV_REQUIRE(M == 0 || (y != nullptr) == (gamma_before != nullptr), NVFP4_ERR_INVALID_ARG,
             "y and gamma_before come together");
  NV_REQUIRE(r_out != r || ldr == K, NVFP4_ERR_MISALIGNED, "in place, r must be contiguous");
  NV_REQUIRE(r_out != r || !stats || M == 0, NVFP4_ERR_INVALID_ARG,
             "stats in place: the backward needs the r that r_out would overwrite");
  NV_REQUIRE(aligned(r_out, 16) && aligned(y, 16) && aligned(stats, 8), NVFP4_ERR_MISALIGNED,
             "r_out and y must be 16-byte aligned");
  const int64_t r_bytes = r_dtype == NVFP4_DT_FP32 ? 4 : 2;
  const int64_t gate_size = gate_kind == NVFP4_GATE_ROW ? M : gate_kind == NVFP4_GATE_CHANNEL ? gate_groups * K : 0;
  st = check_disjoint(__func__, {flat(r_out, M * K, r_bytes), flat(y, M * K, 2), flat(stats, 2 * M, 4)},
                      {{f, M, ldf, K, 2}, {r == r_out ? nullptr : r, M, ldr, K, r_bytes}, flat(gamma_after, K, 2),
                       flat(gamma_before, K, 2), flat(gate, gate_size, 2)});
  if (st != NVFP4_OK) return st;
  DeviceInfo *d;
  if ((st = device_info(__func__, &d)) != NVFP4_OK) return st;
  if (M == 0) return NVFP4_OK;
  NormArgs a = {};
  a.f = f;
  a.r = r;
  a.ldf = ldf;
  a.ldr = ldr;
  a.ldr_out = K;
  a.ga = gamma_after;
  a.gb = gamma_before;
  a.gate = gate;
  a.gate_kind = gate_kind;
  a.rows_per_group = gate_kind == NVFP4_GATE_CHANNEL ? M / gate_groups : M;
  a.scale = scale;
  a.eps = eps;
  a.r_out = r_out;
  a.y = y;
  a.stats = stats;
  a.M = M;
  a.K = static_cast<int>(K);
  a.err = d->flags;
  NV_CUDA(launch_residual_norm(a, dtype, r_dtype == NVFP4_DT_FP32, d->sms, static_cast<cudaStream_t>(stream)),
          "residual norm launch");
  return NVFP4_OK;
}

size_t nvfp4_residual_norm_backward_workspace_bytes(int64_t M, int64_t K, int64_t gate_groups, int r_dtype) {
  if (M < 0 || K <= 0 || K % 8 || K > kNormMaxK || !dims_ok(M, K) || gate_groups < 0) return 0;
  if (M == 0) return 0;
  const int64_t groups = gate_groups > 0 ? gate_groups : 1;
  if (M % groups) return 0;
  const NormGradPlan p = norm_grad_plan(M, K, groups, r_dtype == NVFP4_DT_FP32);
  const size_t rows = static_cast<size_t>(p.ctas) * static_cast<size_t>(K) * 4;
  return 2 * align256(rows) + (p.parts > 1 ? align256(rows) : 0);
}

nvfp4_status nvfp4_residual_norm_backward(const void *dr_out, int64_t lddr, const void *dy, int64_t lddy, const void *f,
                                          int dtype, const void *r, int r_dtype, int64_t M, int64_t K, int64_t ldf,
                                          int64_t ldr, const float *stats, const void *gamma_after, const void *gate,
                                          int gate_kind, int64_t gate_groups, float scale, const void *gamma_before,
                                          void *df, void *dr, float *dgamma_after, float *dgate, float *dgamma_before,
                                          void *ws, size_t ws_bytes, void *stream) {
  nvfp4_status st = check_norm(__func__, f, dtype, r, r_dtype, M, K, ldf, ldr, gamma_after, gate, gate_kind,
                               gate_groups, scale, gamma_before);
  if (st != NVFP4_OK) return st;
  NV_REQUIRE((stats && df && dr) || M == 0, NVFP4_ERR_INVALID_ARG, "NULL pointer argument");
  NV_REQUIRE(gamma_before || !dy, NVFP4_ERR_INVALID_ARG, "dy without gamma_before");
  NV_REQUIRE((gamma_after || !dgamma_after) && (gamma_before || !dgamma_before) && (gate || !dgate),
             NVFP4_ERR_INVALID_ARG, "a gradient of an absent parameter");
  NV_REQUIRE(!dr_out || (lddr >= K && lddr % 8 == 0 && lddr < kMaxDim * 16), NVFP4_ERR_MISALIGNED,
             "lddr=%lld must be >= K and a multiple of 8", (long long)lddr);
  NV_REQUIRE(!dy || (lddy >= K && lddy % 8 == 0 && lddy < kMaxDim * 16), NVFP4_ERR_MISALIGNED,
             "lddy=%lld must be >= K and a multiple of 8", (long long)lddy);
  NV_REQUIRE(aligned(dr_out, 16) && aligned(dy, 16) && aligned(stats, 8) && aligned(df, 16) && aligned(dr, 16) &&
                 aligned(dgamma_after, 16) && aligned(dgamma_before, 16) && aligned(dgate, 16),
             NVFP4_ERR_MISALIGNED, "pointers must be 16-byte aligned");
  const bool channel = gate_kind == NVFP4_GATE_CHANNEL;
  const int64_t groups = channel ? gate_groups : 1;
  const bool r32 = r_dtype == NVFP4_DT_FP32;
  const size_t need = nvfp4_residual_norm_backward_workspace_bytes(M, K, groups, r_dtype);
  if ((st = check_ws(__func__, ws, ws_bytes, need)) != NVFP4_OK) return st;
  const int64_t r_bytes = r32 ? 4 : 2, gate_size = channel ? groups * K : gate ? M : 0;
  st = check_disjoint(__func__,
                      {flat(df, M * K, 2), flat(dr, M * K, r_bytes), flat(dgamma_after, K, 4), flat(dgamma_before, K, 4),
                       flat(dgate, gate_size, 4), flat(ws, static_cast<int64_t>(need), 1)},
                      {{dr_out, M, lddr, K, r_bytes}, {dy, M, lddy, K, 2}, {f, M, ldf, K, 2}, {r, M, ldr, K, r_bytes},
                       flat(stats, 2 * M, 4), flat(gamma_after, K, 2), flat(gamma_before, K, 2), flat(gate, gate_size, 2)});
  if (st != NVFP4_OK) return st;
  DeviceInfo *d;
  if ((st = device_info(__func__, &d)) != NVFP4_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {
    const size_t row = static_cast<size_t>(K) * 4;
    if (dgamma_after) NV_CUDA(cudaMemsetAsync(dgamma_after, 0, row, s), "zero dgamma_after");
    if (dgamma_before) NV_CUDA(cudaMemsetAsync(dgamma_before, 0, row, s), "zero dgamma_before");
    if (dgate && channel) NV_CUDA(cudaMemsetAsync(dgate, 0, row * static_cast<size_t>(groups), s), "zero dgate");
    return NVFP4_OK;
  }
  const NormGradPlan p = norm_grad_plan(M, K, groups, r32);
  const size_t rows = align256(static_cast<size_t>(p.ctas) * static_cast<size_t>(K) * 4);
  uint8_t *w = static_cast<uint8_t *>(ws);
  NormGradArgs a = {};
  a.dr_out = dr_out;
  a.lddr = lddr;
  a.dy = dy;
  a.lddy = lddy;
  a.f = f;
  a.r = r;
  a.ldf = ldf;
  a.ldr = ldr;
  a.stats = stats;
  a.ga = gamma_after;
  a.gb = gamma_before;
  a.gate = gate;
  a.gate_kind = gate_kind;
  a.groups = groups;
  a.rows_per_group = M / groups;
  a.scale = scale;
  a.df = df;
  a.dr = dr;
  a.dga = dgamma_after;
  a.dgb = dgamma_before;
  a.dgate = dgate;
  a.part_a = dgamma_after ? reinterpret_cast<float *>(w) : nullptr;
  a.part_b = dgamma_before ? reinterpret_cast<float *>(w + rows) : nullptr;
  a.part_g = dgate && channel && p.parts > 1 ? reinterpret_cast<float *>(w + 2 * rows) : nullptr;
  a.M = M;
  a.K = static_cast<int>(K);
  a.slices = p.slices;
  a.slice_cols = p.slice_cols;
  a.stages = p.stages;
  a.parts = p.parts;
  a.err = d->flags;
  NV_CUDA(launch_residual_norm_backward(a, p, dtype, r32, s), "residual norm backward launch");
  return NVFP4_OK;
}

}  // extern "C"
