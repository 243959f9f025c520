// Gated linear h = act(x Wg^T) * (x Wu^T) in bf16 or fp16, and its backward pass.
//
// Forward: one kernel makes both products of an output element and applies the activation in its
// epilogue (tile_gemm.cuh for many tokens, stream_gemm.cuh for few).  For training it also leaves
// the pre-activations g and u in fp32: with them the backward needs 8 T H I operations instead of
// the 12 T H I of recomputing g and u, for 8 bytes of memory per element of h, and dg and du carry
// no rounding of g or u.
//
// Backward: dg = dh u act'(g), du = dh act(g) in fp32, rounded once to the operands' 16-bit type as
// tensor-core operands [dg | du]; then dx = dg Wg + du Wu and [dWg; dWu] = [dg | du]^T x, each one
// launch with fp32 accumulators over the whole reduction.
#include "stream_gemm.cuh"
#include "tile_gemm.cuh"

namespace nvfp4 {

namespace {

constexpr int kGbThreads = 256;

// [dg | du] of 8 columns per thread: 10 bytes in and 4 out per element of h, bound by memory
// (4096 x 2048: 16.5 us, 7.1 TB/s, part of it from L2).
template <class T, int kAct>
__global__ void __launch_bounds__(kGbThreads)
    gated_grad_kernel(const uint16_t *__restrict__ dh, int64_t lddh, const float *__restrict__ gu, int64_t M, int I,
                      uint16_t *__restrict__ dgu) {
  pdl_wait();
  pdl_trigger();
  const int chunks = I / 8;
  const int64_t total = M * chunks, step = static_cast<int64_t>(gridDim.x) * kGbThreads;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * kGbThreads + threadIdx.x; e < total; e += step) {
    const int64_t m = e / chunks;
    const int c = static_cast<int>(e - m * chunks) * 8;
    const float4 *gp = reinterpret_cast<const float4 *>(gu + m * 2 * I + c);
    const float4 *up = reinterpret_cast<const float4 *>(gu + m * 2 * I + I + c);
    const uint4 d4 = __ldg(reinterpret_cast<const uint4 *>(dh + m * lddh + c));
    const float4 g0 = __ldcs(gp), g1 = __ldcs(gp + 1), u0 = __ldcs(up), u1 = __ldcs(up + 1);
    const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
    const float u[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
    const uint32_t w[4] = {d4.x, d4.y, d4.z, d4.w};
    uint32_t og[4], ou[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a0, da0, a1, da1;
      act_bwd<kAct>(g[2 * i], a0, da0);
      act_bwd<kAct>(g[2 * i + 1], a1, da1);
      const float d0 = T::lo(w[i]), d1 = T::hi(w[i]);
      og[i] = T::pack(d0 * u[2 * i] * da0, d1 * u[2 * i + 1] * da1);
      ou[i] = T::pack(d0 * a0, d1 * a1);
    }
    *reinterpret_cast<uint4 *>(dgu + m * 2 * I + c) = make_uint4(og[0], og[1], og[2], og[3]);
    *reinterpret_cast<uint4 *>(dgu + m * 2 * I + I + c) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
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
                              void *dgu, int sms, cudaStream_t s) {
  const int64_t blocks = (M * (I / 8) + kGbThreads - 1) / kGbThreads, cap = int64_t(8) * sms;
  const dim3 grid(static_cast<unsigned>(blocks < cap ? blocks : cap));
  NVFP4_BY_ACT(return launch_pdl(dtype == NVFP4_DT_BF16 ? gated_grad_kernel<Bf16, kAct> : gated_grad_kernel<Fp16, kAct>,
                                 grid, dim3(kGbThreads), 0, s, static_cast<const uint16_t *>(dh), lddh, gu, M,
                                 static_cast<int>(I), static_cast<uint16_t *>(dgu)));
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
