// FP8 (e4m3) block-scaled linear: quantisers and the launches of its product.
//
//   activations:  s[b, m] = fl32(max_{k in block b} |x[m, k]| / 448),
//                 q[m, k] = e4m3(fl32(x[m, k] / s[b, m])), 0 where s is 0     (blocks of 128 along K)
//   weights:      the same over 128 x 128 blocks
//   y[m, n]       = sum_b s[b, m] sw[n / 128, b] sum_{k in block b} q[m, k] w[n, k]
//
// Divisions are correctly rounded, so codes and scales are the same on every run and machine that
// divides in IEEE fp32.  A NaN in a block gives a NaN scale (the maximum is taken over the bits of
// |x|, where NaN orders above infinity) and an infinity an infinite one: either way every output of
// that row is NaN, never a finite number made from a dropped NaN.
#include "dense.h"
#include "fp8_encode.cuh"
#include "stream_gemm.cuh"
#include "tile_gemm.cuh"

namespace nvfp4 {

namespace {

constexpr int kFqThreads = 256;
constexpr int kFqGroup = 16;                         // lanes of one 128-element block (8 elements each)
constexpr int kFqRows = kFqThreads / kFqGroup;       // rows of a CTA
constexpr int kFqUnroll = 4;                         // blocks of a row in flight per lane

// One pass over x: a 16-lane group holds one block of one row, 16 rows per CTA, so that the scales
// of a block column leave as 64 consecutive bytes.  2 bytes in and 1 out per element; the encoding's
// instructions take as long as they do (4096 x 7168: 16 us, 5.4 TB/s, issue slots 71% busy; with scalar
// quotients and a division for the scale 20 us).
template <class T>
__global__ void __launch_bounds__(kFqThreads)
    fp8_quantize_act_kernel(const uint16_t *__restrict__ x, int64_t M, int K, int64_t ldx, uint8_t *__restrict__ q,
                            float *__restrict__ s, int64_t lds) {
  pdl_wait();
  pdl_trigger();
  const int gl = threadIdx.x % kFqGroup;
  const int64_t m = static_cast<int64_t>(blockIdx.x) * kFqRows + threadIdx.x / kFqGroup;
  const int blocks = (K + 127) / 128;
  const bool row_ok = m < M;
  for (int b0 = blockIdx.y * kFqUnroll; b0 < blocks; b0 += gridDim.y * kFqUnroll) {
    uint4 v[kFqUnroll];
#pragma unroll
    for (int u = 0; u < kFqUnroll; ++u) {
      const int k = (b0 + u) * 128 + gl * 8;
      v[u] = row_ok && k < K ? __ldg(reinterpret_cast<const uint4 *>(x + m * ldx + k)) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int u = 0; u < kFqUnroll; ++u) {
      uint32_t a = max_abs16(v[u]);
#pragma unroll
      for (int o = kFqGroup / 2; o; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
      const float sc = scale_of<T>(a);
      const int k = (b0 + u) * 128 + gl * 8;
      if (row_ok && k < K) *reinterpret_cast<uint2 *>(q + m * K + k) = encode8<T>(v[u], sc);
      if (row_ok && gl == 0 && b0 + u < blocks) s[(b0 + u) * lds + m] = sc;
    }
  }
}

// One CTA per 128 x 128 block of the weight (once, at load time).
template <class T>
__global__ void __launch_bounds__(kFqThreads)
    fp8_quantize_weight_kernel(const uint16_t *__restrict__ w, int64_t N, int K, int64_t ldw, uint8_t *__restrict__ q,
                               float *__restrict__ s) {
  __shared__ uint32_t red[kFqThreads / 32];
  pdl_wait();
  const int gl = threadIdx.x % kFqGroup, k = blockIdx.x * 128 + gl * 8;
  const int64_t n0 = static_cast<int64_t>(blockIdx.y) * 128 + threadIdx.x / kFqGroup;
  uint4 v[128 / kFqRows];
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 128 / kFqRows; ++i) {
    const int64_t n = n0 + i * kFqRows;
    v[i] = n < N && k < K ? __ldg(reinterpret_cast<const uint4 *>(w + n * ldw + k)) : make_uint4(0u, 0u, 0u, 0u);
    a = max(a, max_abs16(v[i]));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kFqThreads / 32; ++i) a = max(a, red[i]);
  const float sc = scale_of<T>(a);
  if (threadIdx.x == 0) s[static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x] = sc;
#pragma unroll
  for (int i = 0; i < 128 / kFqRows; ++i) {
    const int64_t n = n0 + i * kFqRows;
    if (n < N && k < K) *reinterpret_cast<uint2 *>(q + n * K + k) = encode8<T>(v[i], sc);
  }
}

}  // namespace

cudaError_t launch_fp8_quantize_act(const void *x, int dtype, int64_t M, int64_t K, int64_t ldx, uint8_t *q, float *s,
                                    int64_t lds, int sms, cudaStream_t st) {
  const int64_t rows = (M + kFqRows - 1) / kFqRows, steps = ((K + 127) / 128 + kFqUnroll - 1) / kFqUnroll;
  // enough CTAs for every SM to hold eight: few rows are split along K
  int64_t gy = (8 * sms + rows - 1) / rows;
  if (gy > steps) gy = steps;
  auto kernel = dtype == NVFP4_DT_BF16 ? fp8_quantize_act_kernel<Bf16> : fp8_quantize_act_kernel<Fp16>;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(rows), static_cast<unsigned>(gy)), dim3(kFqThreads), 0, st,
                    static_cast<const uint16_t *>(x), M, static_cast<int>(K), ldx, q, s, lds);
}

cudaError_t launch_fp8_quantize_weight(const void *w, int dtype, int64_t N, int64_t K, int64_t ldw, uint8_t *q,
                                       float *s, cudaStream_t st) {
  auto kernel = dtype == NVFP4_DT_BF16 ? fp8_quantize_weight_kernel<Bf16> : fp8_quantize_weight_kernel<Fp16>;
  const dim3 grid(static_cast<unsigned>((K + 127) / 128), static_cast<unsigned>((N + 127) / 128));
  return launch_pdl(kernel, grid, dim3(kFqThreads), 0, st, static_cast<const uint16_t *>(w), N, static_cast<int>(K),
                    ldw, q, s);
}

cudaError_t launch_fp8_tile_gemm(const CUtensorMap &a, const CUtensorMap &b, const TileArgs &args, int dtype, int cols,
                                 cudaStream_t s) {
  return dtype == NVFP4_DT_BF16 ? launch_tile_gemm_as<TileOp::kFp8, Bf16, 0>(a, a, b, b, a, b, args, cols, s)
                                : launch_tile_gemm_as<TileOp::kFp8, Fp16, 0>(a, a, b, b, a, b, args, cols, s);
}

cudaError_t launch_fp8_stream_gemm(const CUtensorMap &w, const CUtensorMap &x, const StreamArgs &args, int dtype,
                                   int tok, int splits, cudaStream_t s) {
#define NVFP4_TOK(n)                                                                                   \
  case n:                                                                                              \
    return dtype == NVFP4_DT_BF16 ? launch_stream_gemm_as<true, Bf16, 0, n>(w, w, x, args, splits, s) \
                                  : launch_stream_gemm_as<true, Fp16, 0, n>(w, w, x, args, splits, s)
  switch (tok) {
    NVFP4_TOK(16);
    NVFP4_TOK(32);
    NVFP4_TOK(64);
    NVFP4_TOK(128);
  }
#undef NVFP4_TOK
  return cudaErrorInvalidValue;
}

cudaError_t launch_fp8_stream_linear(const CUtensorMap &w, const StreamArgs &args, int dtype, int tok, int splits,
                                     cudaStream_t s) {
#define NVFP4_TOK(n)                                                                                         \
  case n:                                                                                                    \
    return dtype == NVFP4_DT_BF16 ? launch_stream_gemm_as<true, Bf16, 0, n, true>(w, w, w, args, splits, s) \
                                  : launch_stream_gemm_as<true, Fp16, 0, n, true>(w, w, w, args, splits, s)
  switch (tok) {
    NVFP4_TOK(16);
    NVFP4_TOK(32);
  }
#undef NVFP4_TOK
  return cudaErrorInvalidValue;
}

}  // namespace nvfp4
