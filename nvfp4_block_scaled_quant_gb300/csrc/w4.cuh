// Device code shared by the kernels that stream 4-bit weights through the warp-level tensor instructions: a warp takes
// prepared blocks of 64 rows x 128 K out of shared memory and adds their products with 8 or 16 tokens to its sums.
//
//   y = sum over groups of s sum (c - z) x
//
// A code c in the low bits of a bf16 or fp16 number is that number's smallest subnormal times c, and bits 4 to 7 count 16
// times as much (with bit 7 the exponent of a bf16 becomes 1, whose step is the same).  Two masks give the low and high halves
// of a word's even bytes, one shift and the same masks those of the odd ones, and one multiplication and addition of
// each pair takes the zero points off: nine operations for eight codes.  The result (c - z) 2^-kRest is exact in either type and
// normal, so that activations go into the MMA as they are and the sums are multiplied by 2^kRest at the end.  Products are exact,
// sums are fp32, scales apply to the fp32 sums of their group: no weight is rounded.  A group's sum may pass
// fp32's range by 2^kRest.  (In bf16 2^-11 would hold every sum, but those of the smallest activations lose bits that outputs have.)
// (Codes as they are, their sums less z sum x, are five operations, but c x and z x round apart where c = z: under an
// activation of 10^9 times its neighbours, which meets weights of zero, nothing of the neighbours was left.)
#pragma once

#include <atomic>

#include "mma16x8.cuh"
#include "w4.h"

namespace nvfp4 {

// kStep: minus the exponent of the type's smallest subnormal; 2^kUp brings a code to 2^-kRest of its size.
template <class T>
struct W4Scale;
template <>
struct W4Scale<Bf16> {
  static constexpr int kStep = 133, kUp = 126, kRest = kStep - kUp, kMantissa = 7, kBias = 127;
};
template <>
struct W4Scale<Fp16> {
  static constexpr int kStep = 24, kUp = 14, kRest = kStep - kUp, kMantissa = 10, kBias = 15;
};
__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((127 + e) << 23); }
// 2^e in both halves of a word.
template <class T>
__device__ __forceinline__ uint32_t power_of_two2(int e) {
  return static_cast<uint32_t>((e + W4Scale<T>::kBias) << W4Scale<T>::kMantissa) * 0x10001u;
}
template <class T>
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (T::kCode == NVFP4_DT_BF16)
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// D = A B, or D += A B, of 16 x 16 by 16 x 8 with fp32 sums.
template <class T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bool add = true) {
  const float c[4] = {add ? d[0] : 0.f, add ? d[1] : 0.f, add ? d[2] : 0.f, add ? d[3] : 0.f};
  if constexpr (T::kCode == NVFP4_DT_BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

template <class T>
__device__ __forceinline__ uint32_t fma2_16(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  if constexpr (T::kCode == NVFP4_DT_BF16)
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  else
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// -z 2^-kRest in both halves of a word: of zero point z, or of byte j of four of them (at most 15).
template <class T>
__device__ __forceinline__ uint32_t w4_zero(int z) {
  return T::pack(static_cast<float>(-z) * power_of_two(-W4Scale<T>::kRest), static_cast<float>(-z) * power_of_two(-W4Scale<T>::kRest));
}
template <class T>
__device__ __forceinline__ uint32_t w4_zero(uint32_t bytes, int j) {  // under a sign bit a byte is minus its number of subnormal steps
  return mul2<T>(__byte_perm(bytes, 0x80u, 0x4040u + 0x0101u * j), power_of_two2<T>(W4Scale<T>::kUp));
}
// A word of eight codes -> the pairs (c - z) 2^-kRest: low halves of the bytes (elements 0, 1 and 2, 3), high halves (4, 5 and 6, 7).
template <class T>
__device__ __forceinline__ void w4_unpack(uint32_t w, uint32_t zero, uint32_t (&p)[4]) {
  const uint32_t v = w >> 8, low = power_of_two2<T>(W4Scale<T>::kUp), high = power_of_two2<T>(W4Scale<T>::kUp - 4);
  p[0] = fma2_16<T>(w & 0x000F000Fu, low, zero);
  p[1] = fma2_16<T>(v & 0x000F000Fu, low, zero);
  p[2] = fma2_16<T>(w & 0x00F000F0u, high, zero);
  p[3] = fma2_16<T>(v & 0x00F000F0u, high, zero);
}

// A lane's activations of one K block: for each chunk of 32 K and tile of 8 tokens the eight elements 32 c + 8 t .. of
// token g.
template <int kNT>
struct W4Frag {
  uint4 v[4][kNT];
};

// sums += block * x 2^-kRest.  sums[i][n] is the C fragment of row tile i and token tile n, two tokens of a row to a pair.
template <class T, int kGpb, bool kZeros, int kNT>
__device__ __forceinline__ void w4_block(const uint8_t *block, const W4Frag<kNT> &x, uint64_t (&sums)[4][kNT][2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2;
  constexpr int kChunks = 4 / kGpb;  // of a group
#pragma unroll
  for (int gi = 0; gi < kGpb; ++gi) {
#pragma unroll
    for (int pair = 0; pair < 2; ++pair) {  // of row tiles: half as many sums and zero points to hold as with the chunks outside
      float acc[2][kNT][4];  // a group's first MMAs start them
      uint32_t zero[4];      // of rows 32 pair + 8 j + g
      if constexpr (kZeros) {
        const uint32_t zq = *reinterpret_cast<const uint32_t *>(block + kW4CodeBytes + kGpb * 128 + (gi * 8 + g) * 8 + 4 * pair);
#pragma unroll
        for (int j = 0; j < 4; ++j) zero[j] = w4_zero<T>(zq, j);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) zero[j] = w4_zero<T>(8);
      }
#pragma unroll
      for (int cc = 0; cc < kChunks; ++cc) {
        const int c = gi * kChunks + cc;
        const uint4 q = *reinterpret_cast<const uint4 *>(block + ((c * 2 + pair) * 32 + lane) * 16);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t lo[4], hi[4];
          w4_unpack<T>(w[2 * i], zero[2 * i], lo);
          w4_unpack<T>(w[2 * i + 1], zero[2 * i + 1], hi);
          const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
          for (int n = 0; n < kNT; ++n) {
            mma16816<T>(acc[i][n], a0, x.v[c][n].x, x.v[c][n].y, cc != 0);
            mma16816<T>(acc[i][n], a1, x.v[c][n].z, x.v[c][n].w);
          }
        }
      }
      const uint2 sq = *reinterpret_cast<const uint2 *>(block + kW4CodeBytes + (gi * 8 + g) * 16 + 8 * pair);
      const uint32_t sw[2] = {sq.x, sq.y};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float s0 = T::lo(sw[i]), s1 = T::hi(sw[i]);
        const uint64_t s00 = pack_f32x2(s0, s0), s11 = pack_f32x2(s1, s1);
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          uint64_t(&sum)[2] = sums[2 * pair + i][n];
          sum[0] = fma_f32x2(s00, pack_f32x2(acc[i][n][0], acc[i][n][1]), sum[0]);
          sum[1] = fma_f32x2(s11, pack_f32x2(acc[i][n][2], acc[i][n][3]), sum[1]);
        }
      }
    }
  }
}

// A warp's sums in shared memory: token j's 64 rows at j * kW4Pitch (a pitch that spreads the lanes over the banks).
constexpr int kW4Pitch = 68;
template <int kNT>
__device__ __forceinline__ void w4_store_sums(float *at, const uint64_t (&sums)[4][kNT][2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float *row = at + (8 * n + 2 * t) * kW4Pitch + 16 * i + 8 * h + g;
        unpack_f32x2(sums[i][n][h], row[0], row[kW4Pitch]);
      }
}

// The sum over a cluster's CTAs, in their order, of the float at one shared-memory address; every load is in flight before the
// sums.
constexpr int kW4MaxRanks = 8;
__device__ __forceinline__ float cluster_sum(uint32_t at, int ranks) {
  float v[kW4MaxRanks];
#pragma unroll
  for (int r = 0; r < kW4MaxRanks; ++r) {
    v[r] = 0.f;
    if (r < ranks) {
      uint32_t addr;
      asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(at), "r"(r));
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[r]) : "r"(addr) : "memory");
    }
  }
  float sum = v[0];
#pragma unroll
  for (int r = 1; r < kW4MaxRanks; ++r)
    if (r < ranks) sum += v[r];
  return sum;
}

// Lets a kernel have `bytes` of dynamic shared memory, once per device.
template <auto kKernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<bool> ready[64];
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (ready[dev].load()) return cudaSuccess;
  const cudaError_t set = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (set == cudaSuccess) ready[dev].store(true);
  return set;
}

// A launch in clusters of `ranks` CTAs along x that may start while the one before ends.
template <class... KArgs, class... Args>
cudaError_t launch_clusters(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem, int ranks, cudaStream_t s, Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

}  // namespace nvfp4
