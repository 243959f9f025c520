// Device code shared by the kernels that stream 4-bit weights through the warp-level tensor instructions: a warp takes
// prepared blocks of 64 rows x 128 K out of shared memory and adds their products with 8 or 16 tokens to its sums.
//
//   y = sum over groups of s (sum over the group of (c - z) x)
//     = sum over groups of 16 s (sum (1 + c / 16) x - (1 + z / 16) sum x)
//
// (1 + c / 16) is exact in bf16 and fp16 and takes one bit operation per pair of codes beside the shift (the code's bits are
// the top of the mantissa of a number in [1, 2)); taking 8 or z off each weight would cost another one.  sum x of
// each group and token comes from a fifth row tile whose weights are all one.  Products are exact, sums are fp32; the
// difference loses at most about three of fp32's 24 bits, where the result is rounded to 8 or 11.  Scales apply to the
// fp32 sums of their group: no weight is rounded.
#pragma once

#include "mma16x8.cuh"
#include "w4.h"

namespace nvfp4 {

template <class T>
struct W4Bits;
template <>
struct W4Bits<Bf16> {
  static constexpr uint32_t kMask = 0x00780078u, kOne = 0x3F803F80u;
  static constexpr int kRotate = 3;
};
template <>
struct W4Bits<Fp16> {
  static constexpr uint32_t kMask = 0x03C003C0u, kOne = 0x3C003C00u;
  static constexpr int kRotate = 6;
};

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

// A word of eight codes -> (1 + c / 16) of its four pairs.
template <class T>
__device__ __forceinline__ void w4_unpack(uint32_t w, uint32_t (&p)[4]) {
  // written as one operation: with both constants as immediates the compiler takes two (the pair of constants stays in registers)
#pragma unroll
  for (int j = 0; j < 4; ++j)
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;"
        : "=r"(p[j])
        : "r"(j ? __funnelshift_r(w, w, 4 * j) : w), "r"(W4Bits<T>::kMask), "r"(W4Bits<T>::kOne));
}

// A lane's activations of one K block: for each chunk of 32 K and tile of 8 tokens the eight elements 32 c + 8 t .. of
// token g.
template <int kNT>
struct W4Frag {
  uint4 v[4][kNT];
};

// sums += block * x.  sums[i][n] is the C fragment of row tile i and token tile n, two tokens of a row to a pair, without
// the factor 16.
template <class T, int kGpb, bool kZeros, int kNT>
__device__ __forceinline__ void w4_block(const uint8_t *block, const W4Frag<kNT> &x, uint64_t (&sums)[4][kNT][2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2;
  constexpr int kChunks = 4 / kGpb;  // of a group
  const uint32_t ones[4] = {W4Bits<T>::kOne, W4Bits<T>::kOne, W4Bits<T>::kOne, W4Bits<T>::kOne};
#pragma unroll
  for (int gi = 0; gi < kGpb; ++gi) {
    float acc[4][kNT][4], sx[kNT][4];  // a group's first MMAs start them
#pragma unroll
    for (int cc = 0; cc < kChunks; ++cc) {
      const int c = gi * kChunks + cc;
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        mma16816<T>(sx[n], ones, x.v[c][n].x, x.v[c][n].y, cc != 0);
        mma16816<T>(sx[n], ones, x.v[c][n].z, x.v[c][n].w);
      }
#pragma unroll
      for (int pair = 0; pair < 2; ++pair) {
        const uint4 q = *reinterpret_cast<const uint4 *>(block + ((c * 2 + pair) * 32 + lane) * 16);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          uint32_t lo[4], hi[4];
          w4_unpack<T>(w[2 * s], lo);
          w4_unpack<T>(w[2 * s + 1], hi);
          const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
          const int i = 2 * pair + s;
#pragma unroll
          for (int n = 0; n < kNT; ++n) {
            mma16816<T>(acc[i][n], a0, x.v[c][n].x, x.v[c][n].y, cc != 0);
            mma16816<T>(acc[i][n], a1, x.v[c][n].z, x.v[c][n].w);
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
      float z0 = -1.5f, z1 = -1.5f;
      if constexpr (kZeros) {
        const uint32_t zz = zw[i >> 1] >> (16 * (i & 1));
        z0 = -1.f - 0.0625f * static_cast<float>(zz & 0xFFu);
        z1 = -1.f - 0.0625f * static_cast<float>((zz >> 8) & 0xFFu);
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
