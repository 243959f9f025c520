// Launches of the operators on 4-bit weights with group scales (the linear and the mixture-of-experts layer for a few
// tokens), as their C entry points call them, and the layout that the weights are prepared into.
#pragma once

#include "internal.h"

namespace nvfp4 {

// Prepared weights: for each matrix, 64-row panel and 128-wide K block, one contiguous block of
//   4096 bytes of codes   [chunk of 32 K: 4][pair of 16-row tiles: 2][lane: 32][16 bytes],
//   scales (16-bit)       [group of the block: 128 / group][g: 8][row tile i: 4][half h: 2], row 16 i + 8 h + g,
//   zero points (bytes)   in the same order, if the weights have them,
// so that one bulk copy brings everything a warp needs for 64 x 128 weights, and each lane reads its share of the
// m16n8k16 A fragments with 16-byte loads.  A lane (g = lane / 4, t = lane % 4) finds four words of eight codes: K
// elements 32 c + 8 t .. + 7 of rows 32 p + {0, 8, 16, 24} + g.  The order of K inside an MMA is free as long as both
// operands agree, so a word's eight elements are the lane's share of two MMAs: elements 0..3 of the first, 4..7 of
// the second, and the activations need no reordering.  In a word, elements 0 to 7 sit in bits 0, 16, 8, 24, 4, 20, 12 and 28:
// the pairs of the first MMA are the low halves of the bytes, those of the second the high halves.
// Rows and columns that the matrix does not have hold zeros.  A gated matrix (gate rows [0, N / 2), up rows [N / 2, N))
// has 32 gate rows and the 32 up rows of the same outputs in each panel: tiles 0, 1 and 2, 3.
constexpr int kW4PanelRows = 64;
constexpr int kW4BlockK = 128;
constexpr int kW4CodeBytes = kW4PanelRows * kW4BlockK / 2;
constexpr int w4_block_bytes(int groups, bool zeros) { return kW4CodeBytes + kW4PanelRows * groups * (zeros ? 3 : 2); }
inline int64_t w4_panels(int64_t N, bool gated) { return gated ? (N / 2 + 31) / 32 : (N + kW4PanelRows - 1) / kW4PanelRows; }
inline int64_t w4_blocks(int64_t K) { return (K + kW4BlockK - 1) / kW4BlockK; }

cudaError_t launch_w4_prepare(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros, int64_t G, int64_t N,
                              int64_t K, int group, bool gated, uint8_t *out, cudaStream_t s);

struct W4Args {
  const void *x;  // 16-bit (M, K), row stride ldx
  int64_t ldx;
  int M, N, K;
  const uint8_t *w;
  void *y;  // 16-bit (M, N)
  uint32_t *err;
};
// The weight-streaming product of at most 8 * tok8 (16) tokens, K split over a cluster of `splits` CTAs.
cudaError_t launch_w4_stream(const W4Args &a, int dtype, int group, bool zeros, int tok8, int splits, int depth,
                             cudaStream_t s);

// Some ten to some hundred tokens: tokens in tiles of tok (32, 64 or 128), K split over a cluster of `splits` CTAs; x: a map
// of x with boxes of tok rows.
cudaError_t launch_w4_tc(const CUtensorMap &x, const W4Args &a, int dtype, int group, bool zeros, int tok, int splits,
                         cudaStream_t s);

// Many tokens: (c - z) 2^-kRest of the prepared weights as a 16-bit matrix (N, K), the scales as (groups, lds) fp32, and
// the product of that matrix and x on CTA pairs.
struct TileArgs;
cudaError_t launch_w4_expand(const W4Args &a, int dtype, int group, bool zeros, uint16_t *out, float *scales, int64_t lds,
                             cudaStream_t s);
// y: a map of the output with boxes of 32 x 32, used where N % 8 == 0 (else any map).
cudaError_t launch_w4_tile_gemm(const CUtensorMap &w, const CUtensorMap &x, const CUtensorMap &y, const TileArgs &args, int dtype,
                                int group, int cols, cudaStream_t s);

struct W4MoeArgs {
  const void *x;  // 16-bit (T, H), row stride ldx
  int64_t ldx;
  int T, H, I, E, topk;
  const void *router;                           // 16-bit (E, H)
  const uint8_t *w13, *w2, *sh13, *sh2;         // prepared; sh13, sh2 null without a shared expert
  int act;
  void *y;                                      // 16-bit (T, H)
  float *logits;                                // (T, E)
  uint16_t *h;                                  // (rows, I), row t * topk + j, then the shared expert's T rows
  float *part;                                  // (rows, H)
  uint8_t *powers;                              // (rows, panels of h) with row stride ld_powers, fp16: what each panel of h is stored times, as -log2
  int64_t ld_powers;
  int *counters;                                // kW4MoeCounters words and the panels of y, zeroed by the router kernel
  uint32_t *err;
};
constexpr int kW4MoeMaxT = 64, kW4MoeMaxEntries = 512, kW4MoeMaxK = 16;
constexpr int kW4MoeMaxSlots = kW4MoeMaxEntries + kW4MoeMaxT / 8;
constexpr int64_t kW4MoeMaxExperts = 1024, kW4MoeMaxDim = 16384;
// The counters: the item counter on a cache line of its own, the finished panels of h of each slot, the largest power of each row of
// h, and behind them the finished slots of each panel of y.
constexpr int kW4MoeRows = kW4MoeMaxEntries + kW4MoeMaxT;
constexpr int kW4MoeSlotDone = 32, kW4MoeRowPower = kW4MoeSlotDone + kW4MoeMaxSlots, kW4MoeCounters = kW4MoeRowPower + kW4MoeRows;
cudaError_t launch_w4_moe(const W4MoeArgs &a, int dtype, int group, bool zeros, int sms, cudaStream_t s);

}  // namespace nvfp4
