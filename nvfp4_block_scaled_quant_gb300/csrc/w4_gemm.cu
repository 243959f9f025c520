// The linear layer on 4-bit weights for many tokens: the weights are written out once per call as the 16-bit numbers
// (c - z) 2^-kRest (exact), which the CTA-pair GEMM takes as its operand; it applies the scales to each group's fp32 sums.
#include "tile_gemm.cuh"
#include "w4.cuh"

namespace nvfp4 {
namespace {

// One prepared block of 64 x 128 weights per CTA.  Bound by its writes: 7168 x 7168 in about 20 us, 6.5 TB/s.
template <class T, int kGpb, bool kZeros>
__global__ void __launch_bounds__(256) w4_expand_kernel(const uint8_t *w, int N, int K, int blocks, uint16_t *out, float *scales, int64_t lds) {
  constexpr int kBytes = w4_block_bytes(kGpb, kZeros);
  pdl_wait();
  pdl_trigger();
  const int64_t id = blockIdx.x;
  const int b = static_cast<int>(id % blocks), panel = static_cast<int>(id / blocks), tid = threadIdx.x;
  const uint8_t *src = w + id * kBytes;
  const int lane = tid & 31, pair = (tid >> 5) & 1, c = tid >> 6, g = lane >> 2, k = b * kW4BlockK + 32 * c + 8 * (lane & 3);
  const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src) + tid);
  const uint32_t word[4] = {v.x, v.y, v.z, v.w};
  const int gi = c * kGpb / 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = panel * kW4PanelRows + 32 * pair + 8 * i + g;
    uint32_t zero = w4_zero<T>(8), p[4];
    if constexpr (kZeros) zero = w4_zero<T>(__ldg(src + kW4CodeBytes + 128 * kGpb + (gi * 8 + g) * 8 + 4 * pair + i), 0);
    w4_unpack<T>(word[i], zero, p);
    if (row < N && k < K) *reinterpret_cast<uint4 *>(out + static_cast<int64_t>(row) * K + k) = make_uint4(p[0], p[1], p[2], p[3]);
  }
  if (tid < 64 * kGpb) {
    const int at = tid & 63, gj = tid >> 6, row = panel * kW4PanelRows + 16 * ((at >> 1) & 3) + 8 * (at & 1) + (at >> 3);
    const uint16_t s = __ldg(reinterpret_cast<const uint16_t *>(src + kW4CodeBytes) + tid);
    if (row < N && b * kW4BlockK + gj * (kW4BlockK / kGpb) < K) scales[(b * kGpb + gj) * lds + row] = T::up(s);
  }
}

template <class T>
cudaError_t expand_as(const W4Args &a, int group, bool zeros, uint16_t *out, float *scales, int64_t lds, cudaStream_t s) {
  auto kernel = group == 128 ? (zeros ? w4_expand_kernel<T, 1, true> : w4_expand_kernel<T, 1, false>)
                : group == 64 ? (zeros ? w4_expand_kernel<T, 2, true> : w4_expand_kernel<T, 2, false>)
                              : (zeros ? w4_expand_kernel<T, 4, true> : w4_expand_kernel<T, 4, false>);
  const int blocks = static_cast<int>(w4_blocks(a.K));
  return launch_pdl(kernel, dim3(static_cast<unsigned>(w4_panels(a.N, false) * blocks)), dim3(256), 0, s, a.w, a.N, a.K, blocks, out,
                    scales, lds);
}

template <class T>
cudaError_t gemm_as(const CUtensorMap &w, const CUtensorMap &x, const CUtensorMap &y, TileArgs args, int group, int cols, cudaStream_t s) {
  args.factor = static_cast<float>(1 << W4Scale<T>::kRest);
  if (group == 128) return launch_tile_gemm_as<TileOp::kW4, T, 128>(w, w, x, x, y, x, args, cols, s);
  if (group == 64) return launch_tile_gemm_as<TileOp::kW4, T, 64>(w, w, x, x, y, x, args, cols, s);
  return launch_tile_gemm_as<TileOp::kW4, T, 32>(w, w, x, x, y, x, args, cols, s);
}

}  // namespace

cudaError_t launch_w4_expand(const W4Args &a, int dtype, int group, bool zeros, uint16_t *out, float *scales, int64_t lds,
                             cudaStream_t s) {
  return dtype == NVFP4_DT_BF16 ? expand_as<Bf16>(a, group, zeros, out, scales, lds, s) : expand_as<Fp16>(a, group, zeros, out, scales, lds, s);
}

cudaError_t launch_w4_tile_gemm(const CUtensorMap &w, const CUtensorMap &x, const CUtensorMap &y, const TileArgs &args, int dtype,
                                int group, int cols, cudaStream_t s) {
  return dtype == NVFP4_DT_BF16 ? gemm_as<Bf16>(w, x, y, args, group, cols, s) : gemm_as<Fp16>(w, x, y, args, group, cols, s);
}

}  // namespace nvfp4
