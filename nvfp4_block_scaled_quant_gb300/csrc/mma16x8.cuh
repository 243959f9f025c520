// Device primitives of the 8-bit and 16-bit floating-point tensor-core kernels (the FP8
// block-scaled linear and the gated linear): MMA wrappers, instruction descriptors, paired
// TMA loads, packed fp32 arithmetic and typed 16-bit stores.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace nvfp4 {

// ---------------------------------------------------------------- element types

// 16-bit element types by their ABI code (NVFP4_DT_BF16, NVFP4_DT_FP16).
struct Bf16 {
  static constexpr int kCode = NVFP4_DT_BF16;
  static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
  static __device__ __forceinline__ uint16_t one(float a) { return __bfloat16_as_ushort(__float2bfloat16_rn(a)); }
  static __device__ __forceinline__ float up(uint32_t h) { return __uint_as_float(h << 16); }
};
struct Fp16 {
  static constexpr int kCode = NVFP4_DT_FP16;
  static __device__ __forceinline__ float lo(uint32_t w) {
    return __half2float(__ushort_as_half(static_cast<uint16_t>(w)));
  }
  static __device__ __forceinline__ float hi(uint32_t w) {
    return __half2float(__ushort_as_half(static_cast<uint16_t>(w >> 16)));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
  static __device__ __forceinline__ uint16_t one(float a) { return __half_as_ushort(__float2half_rn(a)); }
  static __device__ __forceinline__ float up(uint32_t h) {
    return __half2float(__ushort_as_half(static_cast<uint16_t>(h)));
  }
};

// 16 fp32 values -> 16 elements at dst, of which the first `left` exist; vec: dst is 16-byte aligned.
// A 32-byte aligned dst takes one 256-bit store (a whole sector per lane).
template <class T>
__device__ __forceinline__ void store16(uint16_t *dst, const float (&v)[16], int left, bool vec) {
  if (vec && left >= 16) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = T::pack(v[2 * i], v[2 * i + 1]);
    if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {
      st_global_v8(dst, w);
    } else {
      uint4 *d = reinterpret_cast<uint4 *>(dst);
      d[0] = make_uint4(w[0], w[1], w[2], w[3]);
      d[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < left) dst[i] = T::one(v[i]);
  }
}

// A read-only load that stays where it is written: an ordinary load may be moved down to its first
// use, which undoes a prefetch.
__device__ __forceinline__ float ld_early(const float *p) {
  float v;
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}

// ---------------------------------------------------------------- packed fp32

__device__ __forceinline__ uint64_t pack_f32x2(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t d, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d));
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// ---------------------------------------------------------------- meeting points

// __syncthreads and the cluster barrier for warps that come from role branches: the barrier instructions
// (and the .aligned tensor-memory instructions around them) need converged warps, and the lanes of
// a warp may leave a wait one after the other.
__device__ __forceinline__ void block_meet() {
  __syncwarp();
  __syncthreads();
  __syncwarp();
}
__device__ __forceinline__ void cluster_meet() {
  __syncwarp();
  cluster_sync();
  __syncwarp();
}

// ---------------------------------------------------------------- TMA for a CTA pair

// Load of a box into this CTA's shared memory that completes on `bar_cluster`, a barrier of
// either CTA of the pair given by its shared::cluster address.
__device__ __forceinline__ void tma_load_2d_pair(void *smem_dst, const CUtensorMap *map, int32_t x, int32_t y,
                                                 uint32_t bar_cluster, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(x), "r"(y), "l"(policy)
      : "memory");
}

// ---------------------------------------------------------------- MMA

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(p));
  return p != 0;
}

// Instruction descriptor of kind::f16 and kind::f8f6f4: fp32 accumulator, operand format
// `fmt` on both sides (f16: 0 = fp16, 1 = bf16; f8f6f4: 0 = e4m3), MN-major flags, M and N.
constexpr uint32_t mma_idesc(uint32_t fmt, bool a_mn, bool b_mn, int m, int n) {
  return (1u << 4) | (fmt << 7) | (fmt << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((static_cast<uint32_t>(n) >> 3) << 17) | ((static_cast<uint32_t>(m) >> 4) << 24);
}

// D (+)= A B^T of one 32-byte K step (16 fp16/bf16 or 32 e4m3 elements per row).
template <bool kFp8, bool kPair>
__device__ __forceinline__ void tc_mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
#define NVFP4_MMA(group, kind)                                                                      \
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"                                    \
               "tcgen05.mma.cta_group::" group ".kind::" kind " [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem), \
               "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)                                \
               : "memory")
  if constexpr (kFp8) {
    if constexpr (kPair)
      NVFP4_MMA("2", "f8f6f4");
    else
      NVFP4_MMA("1", "f8f6f4");
  } else {
    if constexpr (kPair)
      NVFP4_MMA("2", "f16");
    else
      NVFP4_MMA("1", "f16");
  }
#undef NVFP4_MMA
}

// ---------------------------------------------------------------- activations of the gated linear

// act(g) = g * p(g) and its derivative in fp32: p is the logistic
// function (SiLU), the normal distribution function (GELU) or the logistic function of
// 2 sqrt(2/pi) (g + 0.044715 g^3), which is (1 + tanh) / 2 of half that argument (tanh GELU).
// Each p is computed without the cancellation of 1 + erf or 1 + tanh at negative g.
//
// The logistic function takes CUDA's fast exponential and division: an error of about 2 + |x| steps of
// 2^-24 of e^-x (which is less than p's share of it for x > 0, and vanishes with g p for x << 0) and two of
// the quotient, far inside the half step of 2^-12 (fp16) that the result is rounded with; exact functions made a
// forward pass of 517 x 1536 x 2048 2 to 4 us longer.  Beyond e^-x = 2^126 the quotient is 0.
__device__ __forceinline__ float logistic(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }
template <int kAct>
__device__ __forceinline__ float act_p(float g) {
  if constexpr (kAct == NVFP4_ACT_SILU) {
    return logistic(g);
  } else if constexpr (kAct == NVFP4_ACT_GELU) {
    return 0.5f * erfcf(-0.70710678118654752f * g);
  } else {
    return logistic(1.59576912160573071f * (g + 0.044715f * g * g * g));
  }
}
template <int kAct>
__device__ __forceinline__ float act_fwd(float g) {
  return g * act_p<kAct>(g);
}
template <int kAct>
__device__ __forceinline__ void act_bwd(float g, float &a, float &da) {
  const float p = act_p<kAct>(g);
  a = g * p;
  if constexpr (kAct == NVFP4_ACT_SILU) {
    da = p + g * p * (1.f - p);
  } else if constexpr (kAct == NVFP4_ACT_GELU) {
    da = p + g * expf(-0.5f * g * g) * 0.39894228040143268f;
  } else {
    // p (1 - p) is 0 long before |g| = 1e4; the square is kept finite, or 0 inf = NaN
    const float b = fminf(fabsf(g), 1e4f);
    da = p + g * p * (1.f - p) * 1.59576912160573071f * (1.f + 0.134145f * b * b);
  }
}

}  // namespace nvfp4
