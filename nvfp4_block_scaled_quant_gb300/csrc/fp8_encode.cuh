// e4m3 block encoding shared by the FP8 quantiser kernels and the streaming GEMM that quantises its own
// activations.
#pragma once

#include "mma16x8.cuh"

namespace nvfp4 {

// The largest |element| of eight 16-bit elements, as bits (NaN orders above infinity).
__device__ __forceinline__ uint32_t max_abs16(const uint4 v) {
  uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
  return max(m & 0xFFFFu, m >> 16);
}

__device__ __forceinline__ uint32_t e4m3x2(uint64_t pair) {
  float a, b;
  unpack_f32x2(pair, a, b);
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3));
}

// fl32(x / s) from r = fl32(1 / s): the product, corrected once by its exact remainder (the last step of
// Markstein's division, "Computation of elementary functions on the IBM RISC System/6000 processor", 1990).
// His proof wants a product within one unit of the last place, which fl32(x r) exceeds for about one pair of
// mantissas in a hundred; that the corrected quotient is the correctly rounded one rests on the operands having few
// bits instead: it holds for every 16-bit mantissa of x with every scale of a 16-bit maximum (16,384
// pairs of bf16 and 1,048,576 of fp16, all of them in the tests).  Powers of two change nothing while the remainder,
// about 2^-24 x, is a normal number: s >= kFastScale and quotients of 2^-12 or more; smaller quotients
// give code 0 either way.
constexpr float kFastScale = 8.2718061e-25f;  // 2^-80
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = __fmul_rn(x, r);
  return __fmaf_rn(__fmaf_rn(-q, s, x), r, q);
}
// The same of two elements at once (minus_s: -s twice, r twice).
__device__ __forceinline__ uint64_t quotients(uint64_t x, uint64_t minus_s, uint64_t r) {
  const uint64_t q = mul_f32x2(x, r);
  return fma_f32x2(fma_f32x2(q, minus_s, x), r, q);
}

// fl32(max / 448) of a 16-bit magnitude given by its bits.  The corrected quotient is right for every
// finite bf16 and fp16 value, subnormal ones included (checked one by one); infinity and NaN stay.
template <class T>
__device__ __forceinline__ float scale_of(uint32_t max_bits) {
  const float a = T::up(max_bits);
  return a < __int_as_float(0x7F800000) ? quotient(a, 448.f, 1.f / 448.f) : a;
}

// 8 elements -> 8 codes
template <class T>
__device__ __forceinline__ uint2 encode8(const uint4 v, float s) {
  if (s == 0.f) return make_uint2(0u, 0u);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
  if (s >= kFastScale && s < __int_as_float(0x7F800000)) {
    const float r = __frcp_rn(s);
    const uint64_t r2 = pack_f32x2(r, r), s2 = pack_f32x2(-s, -s);
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = e4m3x2(quotients(pack_f32x2(T::lo(w[i]), T::hi(w[i])), s2, r2));
  } else {  // tiny, infinite or NaN scales
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = e4m3x2(pack_f32x2(__fdiv_rn(T::lo(w[i]), s), __fdiv_rn(T::hi(w[i]), s)));
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

}  // namespace nvfp4
