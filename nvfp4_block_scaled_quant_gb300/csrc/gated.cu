// Gated linear h = act(x Wg^T) * (x Wu^T) in bf16 or fp16, and its backward pass.
//
// Forward: one kernel makes both products of an output element and applies the activation in its
// epilogue (tile_gemm.cuh for many tokens, stream_gemm.cuh for few).  For training it also leaves
// the pre-activations g and u in fp32: with them the backward needs 8 T H I operations instead of
// the 12 T H I of recomputing g and u, for 8 bytes of memory per element of h, and dg and du carry
// no rounding of g or u.
//
// Backward: dg = dh u act'(g), du = dh act(g) in fp32, rounded once to the operands' 16-bit type as
// tensor-core operands [dg | du]; then dx = dg Wg + du Wu and [dWg; dWu] = [dg | du]^T x in one
// launch, with fp32 accumulators over the whole reduction.  The rounding (half a step of the type per element)
// is the price of 16-bit operands: the gradients' error is 1.4 times that of exact dg and du.
//
// fp16: dg and du may leave the type's range where the gradients do not (a loss-scaled dh of 2000 times u = 50;
// or 1e-5 times 0.1, with two bits left).  So the pair is stored times a power of two that puts its largest
// finite magnitude between 2^14 and 2^15, and the products' epilogue divides it out of the fp32 sums,
// exactly.  An element is then off by half a step or by 2^-39 of the largest one; beside largest gradients of
// 2^16, where the type ends, that is the order of its smallest step, 2^-24.  The maximum takes a pass of its own
// (517 x 2048: 4 us, 4096 x 2048: 9 us); bf16 has fp32's range and needs none.
#include "dense.h"
#include "stream_gemm.cuh"
#include "tile_gemm.cuh"

namespace nvfp4 {

namespace {

constexpr int kGbThreads = 256;

// dg and du of eight columns from dh, g and u at element (m, c).
struct GradOf8 {
  float dg[8], du[8];
};
template <class T, int kAct, bool kLastUse>
__device__ __forceinline__ GradOf8 grad_of8(const uint16_t *dh, int64_t lddh, const float *gu, int I, int64_t m, int c) {
  const float4 *gp = reinterpret_cast<const float4 *>(gu + m * 2 * I + c);
  const float4 *up = reinterpret_cast<const float4 *>(gu + m * 2 * I + I + c);
  const uint4 d4 = __ldg(reinterpret_cast<const uint4 *>(dh + m * lddh + c));
  auto load = [](const float4 *p) { return kLastUse ? __ldcs(p) : __ldg(p); };
  const float4 g0 = load(gp), g1 = load(gp + 1), u0 = load(up), u1 = load(up + 1);
  const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
  const float u[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
  const uint32_t w[4] = {d4.x, d4.y, d4.z, d4.w};
  GradOf8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a, da;
    act_bwd<kAct>(g[i], a, da);
    const float d = (i & 1) ? T::hi(w[i >> 1]) : T::lo(w[i >> 1]);
    r.dg[i] = d * u[i] * da;
    r.du[i] = d * a;
  }
  return r;
}

// fp16: the largest finite |dg|, |du| of each CTA's elements, as bits.  Bound by memory (4096 x 2048: 16.6 us cold,
// about 9 with the forward's outputs still in L2).
template <class T, int kAct>
__global__ void __launch_bounds__(kGbThreads)
    gated_grad_max_kernel(const uint16_t *__restrict__ dh, int64_t lddh, const float *__restrict__ gu, int64_t M, int I,
                          uint32_t *__restrict__ parts) {
  __shared__ uint32_t red[kGbThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int chunks = I / 8;
  const int64_t total = M * chunks, step = static_cast<int64_t>(gridDim.x) * kGbThreads;
  uint32_t most = 0;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * kGbThreads + threadIdx.x; e < total; e += step) {
    const int64_t m = e / chunks;
    const GradOf8 r = grad_of8<T, kAct, false>(dh, lddh, gu, I, m, static_cast<int>(e - m * chunks) * 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t g = __float_as_uint(r.dg[i]) & 0x7FFFFFFFu, u = __float_as_uint(r.du[i]) & 0x7FFFFFFFu;
      most = max(most, max(g < 0x7F800000u ? g : 0u, u < 0x7F800000u ? u : 0u));
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = most;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 1; i < kGbThreads / 32; ++i) most = max(most, red[i]);
    parts[blockIdx.x] = most;
  }
}

// [dg | du] of 8 columns per thread: 10 bytes in and 4 out per element of h, bound by memory
// (4096 x 2048: 18 us, 6.5 TB/s, part of it from L2).  fp16 (parts of the maximum given): times the
// power of two, whose inverse the first CTA leaves in *unscale.
template <class T, int kAct>
__global__ void __launch_bounds__(kGbThreads)
    gated_grad_kernel(const uint16_t *__restrict__ dh, int64_t lddh, const float *__restrict__ gu, int64_t M, int I,
                      uint16_t *__restrict__ dgu, const uint32_t *__restrict__ parts, int part_count,
                      float *__restrict__ unscale) {
  pdl_wait();
  pdl_trigger();
  constexpr bool kScaled = T::kCode == NVFP4_DT_FP16;
  float scale = 1.f;
  if constexpr (kScaled) {
    __shared__ uint32_t red[kGbThreads / 32];
    uint32_t most = 0;
    for (int i = static_cast<int>(threadIdx.x); i < part_count; i += kGbThreads) most = max(most, __ldcg(parts + i));
#pragma unroll
    for (int o = 16; o; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = most;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kGbThreads / 32; ++i) most = max(most, red[i]);
    // biased exponents: the maximum's 127 + e becomes the scale's 127 + 14 - e, both and the inverse normal numbers
    const int field = most == 0u ? 127 : min(127 + 14 + 127 - static_cast<int>(most >> 23), 253);
    scale = __int_as_float(field << 23);
    if (blockIdx.x == 0 && threadIdx.x == 0) *unscale = __int_as_float((254 - field) << 23);
  }
  const int chunks = I / 8;
  const int64_t total = M * chunks, step = static_cast<int64_t>(gridDim.x) * kGbThreads;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * kGbThreads + threadIdx.x; e < total; e += step) {
    const int64_t m = e / chunks;
    const int c = static_cast<int>(e - m * chunks) * 8;
    GradOf8 r = grad_of8<T, kAct, true>(dh, lddh, gu, I, m, c);
    if constexpr (kScaled) {
#pragma unroll
      for (int i = 0; i < 8; ++i) r.dg[i] *= scale, r.du[i] *= scale;
    }
    *reinterpret_cast<uint4 *>(dgu + m * 2 * I + c) =
        make_uint4(T::pack(r.dg[0], r.dg[1]), T::pack(r.dg[2], r.dg[3]), T::pack(r.dg[4], r.dg[5]), T::pack(r.dg[6], r.dg[7]));
    *reinterpret_cast<uint4 *>(dgu + m * 2 * I + I + c) =
        make_uint4(T::pack(r.du[0], r.du[1]), T::pack(r.du[2], r.du[3]), T::pack(r.du[4], r.du[5]), T::pack(r.du[6], r.du[7]));
  }
}

}  // namespace

#define NVFP4_BY_ACT(call)                           \
  switch (act) {                                     \
    case NVFP4_ACT_SILU: { constexpr int kAct = NVFP4_ACT_SILU; call; }             \
    case NVFP4_ACT_GELU: { constexpr int kAct = NVFP4_ACT_GELU; call; }             \
    case NVFP4_ACT_GELU_TANH: { constexpr int kAct = NVFP4_ACT_GELU_TANH; call; }   \
  }                                                  \
  return cudaErrorInvalidValue

cudaError_t launch_gated_grad(const void *dh, int64_t lddh, const float *gu, int64_t M, int64_t I, int dtype, int act,
                              void *dgu, uint32_t *parts, float *unscale, int sms, cudaStream_t s) {
  const int64_t blocks = (M * (I / 8) + kGbThreads - 1) / kGbThreads, cap = int64_t(8) * sms;
  const dim3 grid(static_cast<unsigned>(blocks < cap ? blocks : cap));
  const uint16_t *d = static_cast<const uint16_t *>(dh);
  const int cols = static_cast<int>(I);
  if (dtype == NVFP4_DT_BF16) {
    NVFP4_BY_ACT(return launch_pdl(gated_grad_kernel<Bf16, kAct>, grid, dim3(kGbThreads), 0, s, d, lddh, gu, M, cols,
                                   static_cast<uint16_t *>(dgu), nullptr, 0, nullptr));
  }
  const int count = static_cast<int>(blocks < kGatedGradParts ? blocks : kGatedGradParts);
  auto both = [&](auto max_kernel, auto kernel) {
    const cudaError_t e = launch_pdl(max_kernel, dim3(count), dim3(kGbThreads), 0, s, d, lddh, gu, M, cols, parts);
    return e != cudaSuccess ? e
                            : launch_pdl(kernel, grid, dim3(kGbThreads), 0, s, d, lddh, gu, M, cols,
                                         static_cast<uint16_t *>(dgu), parts, count, unscale);
  };
  NVFP4_BY_ACT(return both(gated_grad_max_kernel<Fp16, kAct>, gated_grad_kernel<Fp16, kAct>));
}

cudaError_t launch_gated_tile_gemm(const CUtensorMap &x, const CUtensorMap &wg, const CUtensorMap &wu,
                                   const TileArgs &args, int dtype, int act, int cols, cudaStream_t s) {
  NVFP4_BY_ACT(return dtype == NVFP4_DT_BF16 ? (launch_tile_gemm_as<TileOp::kGated, Bf16, kAct>(x, x, wg, wu, x, wg, args, cols, s))
                                             : (launch_tile_gemm_as<TileOp::kGated, Fp16, kAct>(x, x, wg, wu, x, wg, args, cols, s)));
}

template <int kTok>
static cudaError_t gated_stream(const CUtensorMap &x, const CUtensorMap &wg, const CUtensorMap &wu,
                                const StreamArgs &args, int dtype, int act, int splits, cudaStream_t s) {
  NVFP4_BY_ACT(return dtype == NVFP4_DT_BF16
                          ? (launch_stream_gemm_as<false, Bf16, kAct, kTok>(wg, wu, x, args, splits, s))
                          : (launch_stream_gemm_as<false, Fp16, kAct, kTok>(wg, wu, x, args, splits, s)));
}

cudaError_t launch_gated_stream_gemm(const CUtensorMap &x, const CUtensorMap &wg, const CUtensorMap &wu,
                                     const StreamArgs &args, int dtype, int act, int tok, int splits, cudaStream_t s) {
  switch (tok) {
    case 16: return gated_stream<16>(x, wg, wu, args, dtype, act, splits, s);
    case 32: return gated_stream<32>(x, wg, wu, args, dtype, act, splits, s);
    case 64: return gated_stream<64>(x, wg, wu, args, dtype, act, splits, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_gated_grad_gemm(const CUtensorMap &dg, const CUtensorMap &du, const CUtensorMap &wg,
                                   const CUtensorMap &wu, const CUtensorMap &dgu, const CUtensorMap &x,
                                   const TileArgs &args, int dtype, int cols, cudaStream_t s) {
  return dtype == NVFP4_DT_BF16 ? launch_tile_gemm_as<TileOp::kGrad, Bf16, 0>(dg, du, wg, wu, dgu, x, args, cols, s)
                                : launch_tile_gemm_as<TileOp::kGrad, Fp16, 0>(dg, du, wg, wu, dgu, x, args, cols, s);
}

}  // namespace nvfp4
