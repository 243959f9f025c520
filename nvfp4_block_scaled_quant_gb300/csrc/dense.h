// Launches of the dense feed-forward operators' kernels (FP8 block-scaled linear, gated linear, residual
// norm), as their C entry points call them.
#pragma once

#include "internal.h"

namespace nvfp4 {

// ---------------------------------------------------------------- FP8 block-scaled linear
struct TileArgs;
struct StreamArgs;
cudaError_t launch_fp8_quantize_act(const void *x, int dtype, int64_t M, int64_t K, int64_t ldx, uint8_t *q, float *s,
                                    int64_t lds, int sms, cudaStream_t st);
cudaError_t launch_fp8_quantize_weight(const void *w, int dtype, int64_t N, int64_t K, int64_t ldw, uint8_t *q,
                                       float *s, cudaStream_t st);
cudaError_t launch_fp8_tile_gemm(const CUtensorMap &a, const CUtensorMap &b, const TileArgs &args, int dtype, int cols,
                                 cudaStream_t s);
cudaError_t launch_fp8_stream_gemm(const CUtensorMap &w, const CUtensorMap &x, const StreamArgs &args, int dtype,
                                   int tok, int splits, cudaStream_t s);
// The same with the activations quantised in the GEMM (args.x, tok 16 or 32).
cudaError_t launch_fp8_stream_linear(const CUtensorMap &w, const StreamArgs &args, int dtype, int tok, int splits,
                                     cudaStream_t s);

// ---------------------------------------------------------------- gated linear
cudaError_t launch_gated_tile_gemm(const CUtensorMap &x, const CUtensorMap &wg, const CUtensorMap &wu,
                                   const TileArgs &args, int dtype, int act, int cols, cudaStream_t s);
cudaError_t launch_gated_stream_gemm(const CUtensorMap &x, const CUtensorMap &wg, const CUtensorMap &wu,
                                     const StreamArgs &args, int dtype, int act, int tok, int splits, cudaStream_t s);
// [dg | du] into dgu.  fp16: times a power of two whose inverse goes to *unscale; parts: kGatedGradParts words.
constexpr int kGatedGradParts = 1024;
cudaError_t launch_gated_grad(const void *dh, int64_t lddh, const float *gu, int64_t M, int64_t I, int dtype, int act,
                              void *dgu, uint32_t *parts, float *unscale, int sms, cudaStream_t s);
cudaError_t launch_gated_grad_gemm(const CUtensorMap &dg, const CUtensorMap &du, const CUtensorMap &wg,
                                   const CUtensorMap &wu, const CUtensorMap &dgu, const CUtensorMap &x,
                                   const TileArgs &args, int dtype, int cols, cudaStream_t s);

// ---------------------------------------------------------------- residual norm
struct NormArgs {
  const void *f, *r;          // (M, K): f 16-bit, r 16-bit or fp32
  int64_t ldf, ldr, ldr_out;  // row strides in elements
  const void *ga, *gb, *gate; // 16-bit, or null
  int gate_kind;
  int64_t rows_per_group;     // rows that share a channel gate
  float scale, eps;
  void *r_out, *y;            // y (M, K) contiguous
  float *stats;               // (M, 2) rstd(f), rstd(r'), or null
  int64_t M;
  int K;
  uint32_t *err;
};
struct NormGradArgs {
  const void *dr_out, *dy;    // or null
  int64_t lddr, lddy;
  const void *f, *r;
  int64_t ldf, ldr;
  const float *stats;
  const void *ga, *gb, *gate;
  int gate_kind;
  int64_t groups, rows_per_group;
  float scale;
  void *df, *dr;              // (M, K) contiguous
  float *dga, *dgb, *dgate;
  float *part_a, *part_b, *part_g;  // per-CTA partial sums
  int64_t M;
  int K;
  int slices, slice_cols, stages, parts;
  uint32_t *err;
};
// Backward launch: ctas x slices CTAs (a cluster of `slices` shares a row), each with a ring of
// `stages` rows; parts: CTAs that share one group of rows (1: a CTA owns whole groups).
struct NormGradPlan {
  int slices, slice_cols, threads, stages, parts, ctas, smem;
};
constexpr int64_t kNormMaxK = 16384;
constexpr int kNormGradThreads = 512; // most threads of a backward CTA: 128 registers each
constexpr int kNormGradGroups = 4;   // groups of four columns of a thread
constexpr int kNormGradMaxCtas = 8;  // most backward CTAs of an SM
constexpr int kNormSlice = 4 * kNormGradGroups * kNormGradThreads;  // columns of a backward CTA
constexpr int kNormMaxSlices = 2;    // ceil(kNormMaxK / kNormSlice)
constexpr int kNormMaxStages = 4;
constexpr int kNormMaxSmem = 225 * 1024;
constexpr int kNormGradRows = 4;     // rows of a backward CTA aimed at when there are few
constexpr int kNormSms = 152;        // the plan must not depend on the device: it sizes the workspace
NormGradPlan norm_grad_plan(int64_t M, int64_t K, int64_t groups, bool r32);
cudaError_t launch_residual_norm(const NormArgs &a, int dtype, bool r32, int sms, cudaStream_t s);
cudaError_t launch_residual_norm_backward(const NormGradArgs &a, const NormGradPlan &p, int dtype, bool r32,
                                          cudaStream_t s);

}  // namespace nvfp4
