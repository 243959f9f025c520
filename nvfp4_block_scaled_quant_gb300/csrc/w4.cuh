// Device code shared by the kernels that stream 4-bit weights through the warp-level tensor instructions: a warp takes
// prepared blocks of 64 rows x 128 K out of shared memory and adds their products with 8 or 16 tokens to its sums.
//
//   y = sum over groups of s (sum (c - z) x) = sum over groups of s (sum c x - z sum x)
//
// A code c in the low bits of a bf16 or fp16 number is that number's smallest subnormal times c, and bits 4 to 7 count 16
// times as much (with bit 7 the exponent of a bf16 becomes 1, whose step is the same): the tensor cores take subnormal operands
// exactly, so the codes need no conversion at all.  Two masks give the low and high halves of a word's even bytes, one
// shift and the same masks those of the odd ones: five operations for eight codes, where numbers 1 + c / 16 took
// seven (these operations bound the product of one token once the weights arrive at the speed of memory: 384 experts, 16
// tokens 445 -> 405 us).  The step of 2^-133 (bf16) or 2^-24 (fp16) is made up for by the activations: a row
// is multiplied by a power of two that brings its largest magnitude to 2^120 (2^14) on its way into the MMA, the elements
// that meet high halves by a sixteenth of it, and the sums by the inverse.  In bf16 nothing is lost by that; in
// fp16 an element keeps everything down to 2^-36 of its row's largest.
// sum x of each group and token comes from a fifth row tile whose codes are all one.  Products are exact, sums are
// fp32, scales apply to the fp32 sums of their group: no weight is rounded.  (A group's sum is 2^-13 of its size in bf16, so that it
// keeps its bits under the smallest scales; brought to 2^60, rows under scales of 2^-76 were 4% off and under 2^-90 zero.)
#pragma once

#include "mma16x8.cuh"
#include "w4.h"

namespace nvfp4 {

// The power of two of a row of activations: kTop - exponent of the largest magnitude, at most kMost; kStep: minus the
// exponent of the smallest subnormal.
template <class T>
struct W4Scale;
template <>
struct W4Scale<Bf16> {
  static constexpr int kTop = 120, kMost = 126, kStep = 133, kMantissa = 7, kBias = 127;
};
template <>
struct W4Scale<Fp16> {
  static constexpr int kTop = 14, kMost = 15, kStep = 24, kMantissa = 10, kBias = 15;
};
// ... from the bits of the row's largest magnitude (infinity and NaN included).
template <class T>
__device__ __forceinline__ int w4_power(uint32_t max_bits) {
  using S = W4Scale<T>;
  return min(S::kTop - (static_cast<int>(max_bits >> S::kMantissa) - S::kBias), S::kMost);
}
__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((127 + e) << 23); }
// A sum of products back in its own size: by 2^(kStep - power) in two steps, which stay in fp32's range.
template <class T>
__device__ __forceinline__ float w4_unscale(float sum, int power) {
  const int e = W4Scale<T>::kStep - power, half = e / 2;
  return sum * power_of_two(half) * power_of_two(e - half);
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

// The largest |element| of eight 16-bit elements, as bits (NaN orders above infinity).
__device__ __forceinline__ uint32_t w4_max_abs(const uint4 v) {
  const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
  return max(m & 0xFFFFu, m >> 16);
}

// A word of eight codes -> its pairs: low halves of the bytes (elements 0, 1 and 2, 3), high halves (4, 5 and 6, 7).
__device__ __forceinline__ void w4_unpack(uint32_t w, uint32_t (&p)[4]) {
  const uint32_t v = w >> 8;
  p[0] = w & 0x000F000Fu;
  p[1] = v & 0x000F000Fu;
  p[2] = w & 0x00F000F0u;
  p[3] = v & 0x00F000F0u;
}

// A lane's activations of one K block: for each chunk of 32 K and tile of 8 tokens the eight elements 32 c + 8 t .. of
// token g.
template <int kNT>
struct W4Frag {
  uint4 v[4][kNT];
};
// The factors of a token's elements, 2^power and a sixteenth of it, in both halves of a word.
struct W4Factor {
  uint32_t low, high;
};
template <class T>
__device__ __forceinline__ W4Factor w4_factor(int power) {
  using S = W4Scale<T>;
  const uint32_t low = static_cast<uint32_t>(power + S::kBias) << S::kMantissa;
  return {low * 0x10001u, (low - (4u << S::kMantissa)) * 0x10001u};
}
template <class T>
__device__ __forceinline__ uint4 w4_scaled(const uint4 v, const W4Factor f) {
  return make_uint4(mul2<T>(v.x, f.low), mul2<T>(v.y, f.low), mul2<T>(v.z, f.high), mul2<T>(v.w, f.high));
}

// sums += block * x with the rows of x multiplied by their powers of two.  sums[i][n] is the C fragment of row tile i and
// token tile n, two tokens of a row to a pair.
template <class T, int kGpb, bool kZeros, int kNT>
__device__ __forceinline__ void w4_block(const uint8_t *block, const W4Frag<kNT> &raw, const W4Factor (&factor)[kNT], uint64_t (&sums)[4][kNT][2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2;
  constexpr int kChunks = 4 / kGpb;  // of a group
  const uint32_t low1[4] = {0x00010001u, 0x00010001u, 0x00010001u, 0x00010001u};
  const uint32_t high1[4] = {0x00100010u, 0x00100010u, 0x00100010u, 0x00100010u};
#pragma unroll
  for (int gi = 0; gi < kGpb; ++gi) {
    float acc[4][kNT][4], sx[kNT][4];  // a group's first MMAs start them
#pragma unroll
    for (int cc = 0; cc < kChunks; ++cc) {
      const int c = gi * kChunks + cc;
      uint4 x[kNT];
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        x[n] = w4_scaled<T>(raw.v[c][n], factor[n]);
        mma16816<T>(sx[n], low1, x[n].x, x[n].y, cc != 0);
        mma16816<T>(sx[n], high1, x[n].z, x[n].w);
      }
#pragma unroll
      for (int pair = 0; pair < 2; ++pair) {
        const uint4 q = *reinterpret_cast<const uint4 *>(block + ((c * 2 + pair) * 32 + lane) * 16);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          uint32_t lo[4], hi[4];
          w4_unpack(w[2 * s], lo);
          w4_unpack(w[2 * s + 1], hi);
          const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
          const int i = 2 * pair + s;
#pragma unroll
          for (int n = 0; n < kNT; ++n) {
            mma16816<T>(acc[i][n], a0, x[n].x, x[n].y, cc != 0);
            mma16816<T>(acc[i][n], a1, x[n].z, x[n].w);
          }
        }
      }
    }
    const uint4 sq = *reinterpret_cast<const uint4 *>(block + kW4CodeBytes + (gi * 8 + g) * 16);
    const uint32_t sw[4] = {sq.x, sq.y, sq.z, sq.w};
    uint32_t zw[2] = {0u, 0u};
    if constexpr (kZeros) {
      const uint2 zq = *reinterpret_cast<const uint2 *>(block + kW4CodeBytes + kGpb * 128 + (gi * 8 + g) * 8);
      zw[0] = zq.x, zw[1] = zq.y;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float s0 = T::lo(sw[i]), s1 = T::hi(sw[i]);
      float z0 = -8.f, z1 = -8.f;
      if constexpr (kZeros) {  // a byte under the exponent of 2^23 is 2^23 + z
        z0 = 8388608.f - __uint_as_float(__byte_perm(zw[i >> 1], 0x4B000000u, 0x7540u + 2 * (i & 1)));
        z1 = 8388608.f - __uint_as_float(__byte_perm(zw[i >> 1], 0x4B000000u, 0x7541u + 2 * (i & 1)));
      }
      const uint64_t s00 = pack_f32x2(s0, s0), s11 = pack_f32x2(s1, s1), z00 = pack_f32x2(z0, z0), z11 = pack_f32x2(z1, z1);
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        const uint64_t sxx = pack_f32x2(sx[n][0], sx[n][1]);
        sums[i][n][0] = fma_f32x2(s00, fma_f32x2(z00, sxx, pack_f32x2(acc[i][n][0], acc[i][n][1])), sums[i][n][0]);
        sums[i][n][1] = fma_f32x2(s11, fma_f32x2(z11, sxx, pack_f32x2(acc[i][n][2], acc[i][n][3])), sums[i][n][1]);
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

}  // namespace nvfp4
