// The boundary between two blocks of a layer in one pass over memory:
//
//   n  = f rstd(f) ga          (the norm after the block; n = f without ga)
//   r' = r + scale gate n      (gate: one value per channel of a group of rows, or one per row)
//   y  = r' rstd(r') gb        (the norm before the next block; from r' before its rounding)
//
// with rstd(v) = 1 / sqrt(mean(v^2) + eps) over a row, all in fp32, and its backward pass.
//
// Backward of one row, with w = ga gate (ga alone for a gate per row), ia = rstd(f), ib = rstd(r'),
// g = scale (times the row's gate), t = w f, rh = ib (r + g ia t) (which is ib r'), v = dy gb,
// u = dr' + ib v, and the sums over the row C2 = sum v rh, A = sum t u, C = sum t rh:
//   kappa = ib C2 / K,  dR = u - kappa rh                the gradient of r' (and of r)
//   S     = sum (ia t) dR = ia (A - kappa C)
//   df    = g ia w dR - (ia f) ia g S / K                (the second term is the norm's)
//   dgate = ga z, dga = gate z with z = sum over rows of g ia dR f; for a gate per row dgate = scale S
//   dgb   = sum over rows of dy rh
// S is linear in dR, so the three sums come from one sweep and one reduction over the block.  No
// power of a statistic is formed: ib^3 and ia^2, gathered out of the sums, leave fp32's range for rows that
// the formulas still handle (ib^3 is zero past an rms of 1e15).
// rstd(f) and rstd(r') are kept by the forward (8 bytes per row); everything else is recomputed.
//
// Both passes are bound by memory: forward f + r in, r' + y out; backward f, r, dr', dy in, df, dr
// out.  Parameter gradients are held in fp32 registers over a CTA's rows (a thread keeps the same 16
// columns), written once per CTA and added in a fixed order by a second kernel: no atomics, so
// repeated calls give identical bits.
#include <atomic>

#include "dense.h"
#include "fp8_encode.cuh"

namespace nvfp4 {

namespace {

// Residual element access: fp32 or the 16-bit type of f, 8 elements at a time.
template <class T, bool kR32>
struct Res {
  static constexpr int kBytes = kR32 ? 4 : 2;
  static __device__ __forceinline__ void load(const void *p, int64_t i, float (&v)[8]) {
    if constexpr (kR32) {
      const float4 *s = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
      const float4 a = s[0], b = s[1];
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      const uint4 a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) v[2 * k] = T::lo(w[k]), v[2 * k + 1] = T::hi(w[k]);
    }
  }
  static __device__ __forceinline__ void store(void *p, int64_t i, const float (&v)[8]) {
    if constexpr (kR32) {
      float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
      d[0] = make_float4(v[0], v[1], v[2], v[3]);
      d[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) =
          make_uint4(T::pack(v[0], v[1]), T::pack(v[2], v[3]), T::pack(v[4], v[5]), T::pack(v[6], v[7]));
    }
  }
};

// Pairs of fp32 values: two elements per instruction, where the number of instructions is what bounds
// a kernel (the many-row kernels: about as many as the memory leaves time for).
struct Two {
  uint64_t v;
};
__device__ __forceinline__ Two two(float a, float b) { return {pack_f32x2(a, b)}; }
__device__ __forceinline__ Two both(float a) { return {pack_f32x2(a, a)}; }
__device__ __forceinline__ Two operator*(Two a, Two b) { return {mul_f32x2(a.v, b.v)}; }
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) { return {fma_f32x2(a.v, b.v, c.v)}; }
__device__ __forceinline__ float sum2(Two a) {
  float x, y;
  unpack_f32x2(a.v, x, y);
  return x + y;
}
template <class T>
__device__ __forceinline__ Two two_of(uint32_t w) {
  return two(T::lo(w), T::hi(w));
}
template <class T>
__device__ __forceinline__ uint32_t pack_two(Two a) {
  float x, y;
  unpack_f32x2(a.v, x, y);
  return T::pack(x, y);
}

// kPairs pairs of elements at element i: fp32, or the 16-bit type T.
template <class T, bool kF32, int kPairs>
__device__ __forceinline__ void load_pairs(const void *p, int64_t i, Two (&v)[kPairs]) {
  if constexpr (kF32) {
#pragma unroll
    for (int k = 0; k < kPairs; k += 2) {
      const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i + 2 * k);
      v[k] = two(a.x, a.y), v[k + 1] = two(a.z, a.w);
    }
  } else if constexpr (kPairs == 2) {
    const uint2 a = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i);
    v[0] = two_of<T>(a.x), v[1] = two_of<T>(a.y);
  } else {
    const uint4 a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
    v[0] = two_of<T>(a.x), v[1] = two_of<T>(a.y), v[2] = two_of<T>(a.z), v[3] = two_of<T>(a.w);
  }
}
template <class T, bool kF32, int kPairs>
__device__ __forceinline__ void store_pairs(void *p, int64_t i, const Two (&v)[kPairs]) {
  if constexpr (kF32) {
#pragma unroll
    for (int k = 0; k < kPairs; k += 2) {
      float4 a;
      unpack_f32x2(v[k].v, a.x, a.y);
      unpack_f32x2(v[k + 1].v, a.z, a.w);
      *reinterpret_cast<float4 *>(static_cast<float *>(p) + i + 2 * k) = a;
    }
  } else if constexpr (kPairs == 2) {
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p) + i) = make_uint2(pack_two<T>(v[0]), pack_two<T>(v[1]));
  } else {
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) =
        make_uint4(pack_two<T>(v[0]), pack_two<T>(v[1]), pack_two<T>(v[2]), pack_two<T>(v[3]));
  }
}
// The same of an optional row vector of parameters: `otherwise` where it is absent.
template <class T, int kPairs>
__device__ __forceinline__ void load_params(const void *p, int64_t i, float otherwise, Two (&v)[kPairs]) {
#pragma unroll
  for (int k = 0; k < kPairs; ++k) v[k] = both(otherwise);
  if (p) load_pairs<T, false, kPairs>(p, i, v);
}

// 8 values of an optional 16-bit row vector, `otherwise` where it is absent.
template <class T>
__device__ __forceinline__ void load_opt(const uint16_t *p, int i, float otherwise, float (&v)[8]) {
  if (p) {
    const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p + i));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) v[2 * k] = T::lo(w[k]), v[2 * k + 1] = T::hi(w[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = otherwise;
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the block in a fixed order; red holds one float per warp and is not reused before the
// next barrier (callers alternate between two).
__device__ __forceinline__ float block_sum(float v, float *red) {
  v = warp_sum(v);
  const int lane = threadIdx.x & 31, warps = static_cast<int>(blockDim.x) >> 5;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(lane < warps ? red[lane] : 0.f);
}

// The group of rows that row m belongs to (row counts are below 2^24).
__device__ __forceinline__ uint32_t group_of(int64_t m, int64_t rows_per_group) {
  return static_cast<uint32_t>(m) / static_cast<uint32_t>(rows_per_group);
}

// rstd of a row over the block, from the thread's part of its sum of squares (red as for block_sum).  The parts
// are scaled by the power of two below 1 / K before they are added, and K alike, so that the sum of a long row
// stays in fp32's range wherever a thread's part does (an rms of 4e18; the sum of 8192 squares only 2e17);
// the bits are those of the plain sum.
__device__ __forceinline__ float row_rstd(float part, float *red, int K, float eps) {
  const float scale = __int_as_float((127 - (32 - __clz(K - 1))) << 23);
  const float mean = __fdiv_rn(block_sum(part * scale, red), static_cast<float>(K) * scale);
  return __fdiv_rn(1.f, __fsqrt_rn(mean + eps));
}

// ---------------------------------------------------------------- 8-bit output

constexpr float kFastMax = 448.f * kFastScale;
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Eight columns of y in e4m3: the scale is max|y| / 448 over the 128 columns that 16 consecutive lanes hold, from y before
// its rounding to 16 bits (rounded once, from fp32, the codes are the nearest ones; a quantiser behind the 16-bit output
// rounds twice).  Lanes without columns pass zeros.  The corrected quotient is within a step of fp32, which can only decide
// between codes at a midpoint.  A NaN stays in the maximum and makes the scale NaN.
__device__ __forceinline__ uint2 encode_columns(const Two (&v)[4], float &scale) {
  float f[8], m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    unpack_f32x2(v[i].v, f[2 * i], f[2 * i + 1]);
    m = max_nan(m, max_nan(fabsf(f[2 * i]), fabsf(f[2 * i + 1])));
  }
#pragma unroll
  for (int o = 8; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  uint32_t c[4];
  if (m >= kFastMax && m < __int_as_float(0x7F800000)) {
    // fl32(m / 448) by the corrected product: right for every mantissa (all of them in the tests)
    scale = quotient(m, 448.f, 1.f / 448.f);
    float rcp;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rcp) : "f"(scale));
    const Two r = both(rcp), minus = both(-scale);
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = e4m3x2(quotients(v[i].v, minus.v, r.v));
  } else {  // zero, tiny, infinite or NaN maxima
    scale = __fdiv_rn(m, 448.f);
    if (scale == 0.f) return make_uint2(0u, 0u);
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = e4m3x2(pack_f32x2(__fdiv_rn(f[2 * i], scale), __fdiv_rn(f[2 * i + 1], scale)));
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}
// The same into the arrays: chunk c (eight columns) of row m.
__device__ __forceinline__ void store_columns8(const NormArgs &a, int64_t m, int c, bool live, const Two (&v)[4]) {
  float scale;
  const uint2 code = encode_columns(v, scale);
  if (live) {
    *reinterpret_cast<uint2 *>(a.q + m * a.K + c * 8) = code;
    if ((c & 15) == 0) a.s[(c >> 4) * a.lds + m] = scale;
  }
}

// ---------------------------------------------------------------- forward

// Few rows: one row per CTA, kChunks groups of 8 columns per thread, in registers over both
// reductions.  kOut8: y in 8 bits, and in 16 if a.y is given (one row of 7168 3.3 us).
template <class T, bool kR32, int kChunks, bool kOut8>
__global__ void __launch_bounds__(1024, 1) residual_norm_kernel(const NormArgs a) {
  __shared__ float red[2][32];
  pdl_wait();
  pdl_trigger();
  const int chunks = a.K / 8, nt = static_cast<int>(blockDim.x);
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const uint16_t *f = static_cast<const uint16_t *>(a.f) + m * a.ldf;
    const uint16_t *gate = static_cast<const uint16_t *>(a.gate);
    float gm = a.scale;
    if (a.gate_kind == NVFP4_GATE_ROW) {
      gm *= T::up(__ldg(gate + m));
      gate = nullptr;
    } else if (gate) {
      gate += static_cast<int64_t>(group_of(m, a.rows_per_group)) * a.K;
    }
    uint4 fv[kChunks];
    float rv[kChunks][8];
    float s = 0.f;
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
      const int c = static_cast<int>(threadIdx.x) + u * nt;
      fv[u] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int i = 0; i < 8; ++i) rv[u][i] = 0.f;
      if (c < chunks) {
        fv[u] = *reinterpret_cast<const uint4 *>(f + c * 8);
        Res<T, kR32>::load(a.r, m * a.ldr + c * 8, rv[u]);
      }
    }
    float ia = 1.f;
    if (a.ga) {
#pragma unroll
      for (int u = 0; u < kChunks; ++u) {
        const uint32_t w[4] = {fv[u].x, fv[u].y, fv[u].z, fv[u].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float lo = T::lo(w[i]), hi = T::hi(w[i]);
          s += lo * lo;
          s += hi * hi;
        }
      }
      ia = row_rstd(s, red[0], a.K, a.eps);
    }
    s = 0.f;
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
      const int c = static_cast<int>(threadIdx.x) + u * nt;
      if (c < chunks) {
        float ga[8], gk[8];
        load_opt<T>(static_cast<const uint16_t *>(a.ga), c * 8, 1.f, ga);
        load_opt<T>(gate, c * 8, 1.f, gk);
        const uint32_t w[4] = {fv[u].x, fv[u].y, fv[u].z, fv[u].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = (i & 1) ? T::hi(w[i >> 1]) : T::lo(w[i >> 1]);
          rv[u][i] += gm * gk[i] * (x * ia * ga[i]);
          s += rv[u][i] * rv[u][i];
        }
        Res<T, kR32>::store(a.r_out, m * a.ldr_out + c * 8, rv[u]);
      }
    }
    float ib = 0.f;
    if (a.gb) {
      ib = row_rstd(s, red[1], a.K, a.eps);
#pragma unroll
      for (int u = 0; u < kChunks; ++u) {
        const int c = static_cast<int>(threadIdx.x) + u * nt;
        if (kOut8 || c < chunks) {
          float gb[8], y[8];
          load_opt<T>(kOut8 && c >= chunks ? nullptr : static_cast<const uint16_t *>(a.gb), c * 8, 1.f, gb);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = rv[u][i] * ib * gb[i];
          if (!kOut8 || (c < chunks && a.y)) Res<T, false>::store(a.y, m * a.K + c * 8, y);
          if constexpr (kOut8) {
            const Two v[4] = {two(y[0], y[1]), two(y[2], y[3]), two(y[4], y[5]), two(y[6], y[7])};
            store_columns8(a, m, c, c < chunks, v);
          }
        }
      }
    }
    if (a.stats && threadIdx.x == 0) *reinterpret_cast<float2 *>(a.stats + 2 * m) = make_float2(a.ga ? ia : 0.f, ib);
    __syncthreads();  // red is reused by the next row
  }
}

// Many rows: each CTA walks its rows through a ring in shared memory (one bulk copy per row and
// tensor), so the next rows load while this one passes its two reductions.  16 columns per thread
// and two CTAs per SM at most widths: one CTA's reductions overlap the other's.
// kThreads, kCtas: most threads of a CTA and CTAs per SM, which set the registers per thread: the
// parameters of a thread's columns stay in registers (the ring leaves little of the SM's memory to
// its cache, and re-reading them for every row cost as much as the rows).  8192 x 7168 in bf16: 76 us,
// 6.2 TB/s; 4096 x 7168 with both outputs (kOut8) 47.7 us, 5.6 TB/s, 70% of the issue slots.
template <class T, bool kR32, int kChunks, int kThreads, int kCtas, bool kOut8>
__global__ void __launch_bounds__(kThreads, kCtas) residual_norm_rows_kernel(const NormArgs a, int stages) {
  extern __shared__ __align__(128) uint8_t smem[];  // used as declared: its loads are known to be shared ones
  __shared__ float red[2][32];
  __shared__ uint64_t full[kNormMaxStages];
  __shared__ int s_abort;
  volatile int *abort_flag = &s_abort;
  const int chunks = a.K / 8, nt = static_cast<int>(blockDim.x), tid = static_cast<int>(threadIdx.x);
  const uint32_t n16 = static_cast<uint32_t>(a.K) * 2u, nr = static_cast<uint32_t>(a.K) * Res<T, kR32>::kBytes;
  const uint32_t stage_bytes = n16 + nr;
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
    s_abort = 0;
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const uint64_t pol = policy_evict_first();
  auto load_row = [&](int64_t m, int s) {
    mbar_arrive_expect_tx(&full[s], stage_bytes);
    uint8_t *d = smem + s * stage_bytes;
    bulk_load(d, static_cast<const uint16_t *>(a.f) + m * a.ldf, n16, &full[s], pol);
    bulk_load(d + n16, static_cast<const uint8_t *>(a.r) + m * a.ldr * Res<T, kR32>::kBytes, nr, &full[s], pol);
  };
  const int64_t step = gridDim.x;
  if (tid == 0)
    for (int s = 0; s < stages && blockIdx.x + s * step < a.M; ++s) load_row(blockIdx.x + s * step, s);
  int s = 0;
  uint32_t phase = 0;
  const uint16_t *gate0 = static_cast<const uint16_t *>(a.gate);
  const bool channel_gate = a.gate_kind == NVFP4_GATE_CHANNEL;
  // w = ga gate and gb of the thread's columns: r' = r + (scale rstd(f)) w f, y = (rstd(r') r') gb
  Two w[kChunks][4], gb[kChunks][4];
  auto load_w = [&](int64_t g) {
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
      const int c = tid + u * nt;
      Two gate[4];
      const bool live = c < chunks;
      load_params<T, 4>(live ? a.ga : nullptr, c * 8, 1.f, w[u]);
      load_params<T, 4>(live && channel_gate ? gate0 + g * a.K : nullptr, c * 8, 1.f, gate);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[u][i] = w[u][i] * gate[i];
    }
  };
  load_w(0);
#pragma unroll
  for (int u = 0; u < kChunks; ++u)
    load_params<T, 4>(tid + u * nt < chunks ? a.gb : nullptr, (tid + u * nt) * 8, 1.f, gb[u]);
  int64_t group = 0;
  float next_gm = a.gate_kind == NVFP4_GATE_ROW && blockIdx.x < a.M ? T::up(__ldg(gate0 + blockIdx.x)) : 1.f;
  for (int64_t m = blockIdx.x; m < a.M; m += step) {
    const float gm = a.scale * next_gm;
    if (a.gate_kind == NVFP4_GATE_ROW && m + step < a.M) next_gm = T::up(__ldg(gate0 + m + step));
    if (channel_gate) {
      const int64_t g = group_of(m, a.rows_per_group);
      if (g != group) {
        group = g;
        load_w(g);
      }
    }
    // a wait that gives up raises the fault flag; every barrier below is still met
    mbar_wait_bounded(&full[s], phase, abort_flag, a.err, kPipelineTimeoutNs);
    const uint8_t *d = smem + s * stage_bytes;
    Two v[kChunks][4];
    Two sum = both(0.f);
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
      const int c = tid + u * nt;
      if (c < chunks) {
        load_pairs<T, false, 4>(d, c * 8, v[u]);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum = fma2(v[u][i], v[u][i], sum);
      }
    }
    const float ia = a.ga ? row_rstd(sum2(sum), red[0], a.K, a.eps) : 1.f;
    const Two c1 = both(gm * ia);
    sum = both(0.f);
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
      const int c = tid + u * nt;
      if (c < chunks) {
        Two x[4];
        load_pairs<T, kR32, 4>(d + n16, c * 8, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[u][i] = fma2(c1, v[u][i] * w[u][i], x[i]);
          sum = fma2(v[u][i], v[u][i], sum);
        }
        store_pairs<T, kR32, 4>(a.r_out, m * a.ldr_out + c * 8, v[u]);
      }
    }
    float ib = 0.f;
    if (a.gb) {
      ib = row_rstd(sum2(sum), red[1], a.K, a.eps);  // its barrier: every thread has read the stage
    } else {
      __syncthreads();
    }
    if (tid == 0 && m + stages * step < a.M) load_row(m + stages * step, s);
    if (++s == stages) {
      s = 0;
      phase ^= 1;
    }
    if (a.gb) {
#pragma unroll
      for (int u = 0; u < kChunks; ++u) {
        const int c = tid + u * nt;
        if (c < chunks) {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[u][i] = (v[u][i] * both(ib)) * gb[u][i];
          if (!kOut8 || a.y) store_pairs<T, false, 4>(a.y, m * a.K + c * 8, v[u]);
        }
        if constexpr (kOut8) {
          if (c >= chunks) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[u][i] = both(0.f);
          }
          store_columns8(a, m, c, c < chunks, v[u]);
        }
      }
      // red[1] is written again only after the next row's first barrier, or this one without ga
      if (!a.ga) __syncthreads();
    }
    if (a.stats && tid == 0) *reinterpret_cast<float2 *>(a.stats + 2 * m) = make_float2(a.ga ? ia : 0.f, ib);
  }
  if (*abort_flag) {  // copies in flight land before the CTA's memory goes
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 10000000ull) {
    }
  }
}

// ---------------------------------------------------------------- backward

// Rows stream through a ring in shared memory (one bulk copy per row and tensor), so the next rows
// load while this one is reduced; registers hold the parameter gradients of a thread's 16 columns.  A
// row of more than kNormSlice columns is split over the CTAs of a cluster, which exchange the three sums.
//
// Half of the time of a 16-bit row is instructions (two sweeps over the row, 16 conversions per four
// columns), so sums go in packed fp32, a thread takes 16 columns (its fixed work per row, two
// reductions and a wait, is spread over more than with 8: 384 instructions per eight columns; about 90
// more with 8), and the warp that is last to finish a row's stage refills it.  8192 x 7168: bf16 139 us, 5.1 TB/s; with an
// fp32 residual 143 us, 7.4 TB/s.  Measured and left: sums of the next row taken while this row's are
// exchanged (147 us: one row fewer is loading), scalar fp32 (144 us).
constexpr int kNbRedFloats = 4 * 32;  // three sums of up to 32 warps each, and a row of zeros

template <class T, bool kR32>
__global__ void __launch_bounds__(kNormGradThreads, 1) residual_norm_backward_kernel(const NormGradArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];  // used as declared: its loads are known to be shared ones
  __shared__ __align__(16) float red[2][kNbRedFloats];
  __shared__ float peer_sums[2][kNormMaxSlices][3];
  __shared__ uint64_t full[kNormMaxStages];
  __shared__ unsigned done[kNormMaxStages];  // warps done with the stage
  __shared__ int s_abort;
  volatile int *abort_flag = &s_abort;

  const int slice = static_cast<int>(blockIdx.x) % a.slices, part = static_cast<int>(blockIdx.x) / a.slices;
  const int k0 = slice * a.slice_cols, cols = min(a.slice_cols, a.K - k0);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // this thread's columns of the slice: groups of four, each contiguous over the block
  int col[kNormGradGroups];
  bool live[kNormGradGroups];
#pragma unroll
  for (int h = 0; h < kNormGradGroups; ++h) {
    col[h] = static_cast<int>(blockDim.x * h + threadIdx.x) * 4;
    live[h] = col[h] < cols;
  }
  // ring stage: f, dy (16 bits), r, dr' (16 or 32 bits), each slice_cols wide
  const int b16 = a.slice_cols * 2, br = a.slice_cols * Res<T, kR32>::kBytes;
  const int stage_bytes = 2 * b16 + 2 * br;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) mbar_init(&full[s], 1), done[s] = 0;
    s_abort = 0;
    fence_barrier_init();
  }
  for (int i = static_cast<int>(threadIdx.x); i < 2 * kNbRedFloats; i += static_cast<int>(blockDim.x)) red[0][i] = 0.f;
  // an absent gradient reads as zeros: no copy touches its part of the stages
  for (int s = 0; s < a.stages; ++s) {
    uint4 *d = reinterpret_cast<uint4 *>(smem + s * stage_bytes);
    for (int i = static_cast<int>(threadIdx.x); i < b16 / 16 && !a.dy; i += static_cast<int>(blockDim.x))
      d[b16 / 16 + i] = make_uint4(0u, 0u, 0u, 0u);
    for (int i = static_cast<int>(threadIdx.x); i < br / 16 && !a.dr_out; i += static_cast<int>(blockDim.x))
      d[(2 * b16 + br) / 16 + i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __syncthreads();
  if (a.slices > 1) cluster_meet();  // the other slices' memory may be written from here on
  pdl_wait();
  pdl_trigger();

  // rows of this CTA: a share of one group of rows (parts > 1), or a range of whole groups
  int64_t m_first, m_last;
  if (a.parts > 1) {
    const int64_t g = part / a.parts, p = part % a.parts;
    m_first = g * a.rows_per_group + a.rows_per_group * p / a.parts;
    m_last = g * a.rows_per_group + a.rows_per_group * (p + 1) / a.parts;
  } else {
    const int64_t ctas = gridDim.x / a.slices;
    m_first = a.groups * part / ctas * a.rows_per_group;
    m_last = a.groups * (part + 1) / ctas * a.rows_per_group;
  }
  const uint64_t pol = policy_evict_first();
  auto load_row = [&](int64_t m, int s) {
    uint8_t *d = smem + s * stage_bytes;
    const uint32_t n16 = static_cast<uint32_t>(cols) * 2u, nr = static_cast<uint32_t>(cols) * Res<T, kR32>::kBytes;
    mbar_arrive_expect_tx(&full[s], n16 + nr + (a.dy ? n16 : 0u) + (a.dr_out ? nr : 0u));
    bulk_load(d, static_cast<const uint16_t *>(a.f) + m * a.ldf + k0, n16, &full[s], pol);
    bulk_load(d + 2 * b16, static_cast<const uint8_t *>(a.r) + (m * a.ldr + k0) * Res<T, kR32>::kBytes, nr, &full[s], pol);
    if (a.dy) bulk_load(d + b16, static_cast<const uint16_t *>(a.dy) + m * a.lddy + k0, n16, &full[s], pol);
    if (a.dr_out)
      bulk_load(d + 2 * b16 + br, static_cast<const uint8_t *>(a.dr_out) + (m * a.lddr + k0) * Res<T, kR32>::kBytes, nr,
                &full[s], pol);
  };
  if (threadIdx.x == 0)
    for (int s = 0; s < a.stages && m_first + s < m_last; ++s) load_row(m_first + s, s);

  const uint16_t *gp = static_cast<const uint16_t *>(a.gate);
  const bool row_gate = a.gate_kind == NVFP4_GATE_ROW, channel_gate = a.gate_kind == NVFP4_GATE_CHANNEL;
  const float inv_k = 1.f / static_cast<float>(a.K);
  // Per thread and column: w = ga gate (it changes with the group of rows) and gb; the sums over rows
  // of dy rh (dgb) and z = g ia dR f, of which both dga = gate z and dgate = ga z are multiples.
  Two w[kNormGradGroups][2], gb[kNormGradGroups][2];
  Two acc_a[kNormGradGroups][2], acc_b[kNormGradGroups][2], acc_z[kNormGradGroups][2];
#pragma unroll
  for (int h = 0; h < kNormGradGroups; ++h) {
    load_params<T, 2>(live[h] ? a.gb : nullptr, k0 + col[h], 0.f, gb[h]);
    if (!a.gb) gb[h][0] = gb[h][1] = both(0.f);
#pragma unroll
    for (int i = 0; i < 2; ++i) acc_a[h][i] = acc_b[h][i] = acc_z[h][i] = both(0.f);
  }
  int64_t group = 0;
  int64_t rows_left = 0;  // rows of the current group still to come, this one included
  int s = 0;
  uint32_t phase = 0;
  // a row's statistics and gate are fetched one row ahead
  float2 next_st = make_float2(0.f, 0.f);
  float next_gate = 1.f;
  auto fetch_row = [&](int64_t m) {
    next_st = __ldg(reinterpret_cast<const float2 *>(a.stats) + m);
    if (row_gate) next_gate = T::up(__ldg(gp + m));
  };
  if (m_first < m_last) fetch_row(m_first);

  for (int64_t m = m_first; m < m_last; ++m) {
    const int pb = static_cast<int>((m - m_first) & 1);
    const float ia = a.ga ? next_st.x : 1.f, ib = next_st.y, gm = a.scale * next_gate;
    if (m + 1 < m_last) fetch_row(m + 1);
    if (rows_left == 0) {  // the first row of this CTA or of a group
      group = group_of(m, a.rows_per_group);
      rows_left = min((group + 1) * a.rows_per_group, m_last) - m;
#pragma unroll
      for (int h = 0; h < kNormGradGroups; ++h) {
        Two gate[2];
        load_params<T, 2>(live[h] ? a.ga : nullptr, k0 + col[h], 1.f, w[h]);
        load_params<T, 2>(live[h] && channel_gate ? gp + group * a.K : nullptr, k0 + col[h], 1.f, gate);
        w[h][0] = w[h][0] * gate[0];
        w[h][1] = w[h][1] * gate[1];
      }
    }
    --rows_left;
    // a wait that gives up leaves this CTA's results undefined and the fault flag raised, but every
    // barrier below is still met
    mbar_wait_bounded(&full[s], phase, abort_flag, a.err, kPipelineTimeoutNs);
    const uint8_t *d = smem + s * stage_bytes;
    const Two c1 = both(gm * ia), ib2 = both(ib);
    Two fv[2], tv[2], rv[2], dyv[2], uv[2];  // f, t, rh, dy and dr' of four columns
    auto fetch = [&](int h) {
      load_pairs<T, false, 2>(d, col[h], fv);
      load_pairs<T, kR32, 2>(d + 2 * b16, col[h], rv);
      load_pairs<T, false, 2>(d + b16, col[h], dyv);
      load_pairs<T, kR32, 2>(d + 2 * b16 + br, col[h], uv);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        tv[i] = fv[i] * w[h][i];
        rv[i] = ib2 * fma2(c1, tv[i], rv[i]);
      }
    };
    Two s2 = both(0.f), sA = both(0.f), sC = both(0.f);
#pragma unroll
    for (int h = 0; h < kNormGradGroups; ++h) {
      if (live[h]) {
        fetch(h);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const Two v = dyv[i] * gb[h][i];
          s2 = fma2(v, rv[i], s2);
          sA = fma2(tv[i], fma2(ib2, v, uv[i]), sA);
          sC = fma2(tv[i], rv[i], sC);
        }
      }
    }
    float c2 = sum2(s2), sa = sum2(sA), sc = sum2(sC);
    // the three sums over the block: lanes 8 j .. 8 j + 7 carry sum j from the second step on
    {
      const bool up16 = lane & 16, up8 = lane & 8;
      const float x = up16 ? c2 : sc, y = up16 ? sa : 0.f;
      float lo = (up16 ? sc : c2) + __shfl_xor_sync(0xffffffffu, x, 16);
      float hi = (up16 ? 0.f : sa) + __shfl_xor_sync(0xffffffffu, y, 16);
      float t = (up8 ? hi : lo) + __shfl_xor_sync(0xffffffffu, up8 ? lo : hi, 8);
#pragma unroll
      for (int o = 4; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      if ((lane & 7) == 0) red[pb][(lane >> 3) * 32 + warp] = t;
    }
    __syncthreads();
    {
      const float4 v = *reinterpret_cast<const float4 *>(&red[pb][lane * 4]);
      float t = (v.x + v.y) + (v.z + v.w);
#pragma unroll
      for (int o = 4; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      c2 = __shfl_sync(0xffffffffu, t, 0);
      sa = __shfl_sync(0xffffffffu, t, 8);
      sc = __shfl_sync(0xffffffffu, t, 16);
    }
    if (a.slices > 1) {  // the other slices' sums, by rank
      if (threadIdx.x < static_cast<unsigned>(a.slices)) {
        const uint32_t at = cluster_addr(&peer_sums[pb][slice][0], threadIdx.x);
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(c2) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at + 4), "f"(sa) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at + 8), "f"(sc) : "memory");
      }
      cluster_meet();
      c2 = sa = sc = 0.f;
      for (int r = 0; r < a.slices; ++r) {
        c2 += peer_sums[pb][r][0];
        sa += peer_sums[pb][r][1];
        sc += peer_sums[pb][r][2];
      }
    }
    const float kappa = ib * (c2 * inv_k);
    const float S = ia * (sa - kappa * sc);
    const Two nk = both(-kappa), nl = both(a.ga ? -ia * (gm * (S * inv_k)) : 0.f), ia2 = both(ia);
    if (row_gate && a.dgate && threadIdx.x == 0 && slice == 0) a.dgate[m] = a.scale * S;
#pragma unroll
    for (int h = 0; h < kNormGradGroups; ++h) {
      if (live[h]) {
        fetch(h);
        Two df[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          acc_b[h][i] = fma2(dyv[i], rv[i], acc_b[h][i]);
          uv[i] = fma2(nk, rv[i], fma2(ib2, dyv[i] * gb[h][i], uv[i]));
          const Two sdr = c1 * uv[i];
          acc_z[h][i] = fma2(sdr, fv[i], acc_z[h][i]);
          df[i] = fma2(nl, ia2 * fv[i], sdr * w[h][i]);
        }
        store_pairs<T, kR32, 2>(a.dr, m * a.K + k0 + col[h], uv);
        store_pairs<T, false, 2>(a.df, m * a.K + k0 + col[h], df);
      }
    }
    // the last warp that is done with the stage fills it again (the counter returns to zero)
    __syncwarp();
    if (lane == 0) {
      __threadfence_block();
      if (atomicInc(&done[s], (blockDim.x >> 5) - 1) == (blockDim.x >> 5) - 1 && m + a.stages < m_last) {
        __threadfence_block();
        load_row(m + a.stages, s);
      }
    }
    if (rows_left == 0) {  // the end of a group of rows
      const int64_t at = (a.parts > 1 ? part : group) * a.K + k0;
#pragma unroll
      for (int h = 0; h < kNormGradGroups; ++h) {
        if (live[h]) {
          Two x[2], gate[2];
          load_params<T, 2>(channel_gate ? gp + group * a.K : nullptr, k0 + col[h], 1.f, gate);
          load_params<T, 2>(a.ga, k0 + col[h], 1.f, x);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            acc_a[h][i] = fma2(gate[i], acc_z[h][i], acc_a[h][i]);
            x[i] = x[i] * acc_z[h][i];
            acc_z[h][i] = both(0.f);
          }
          if (channel_gate && a.dgate) store_pairs<T, true, 2>((a.parts > 1 ? a.part_g : a.dgate) + at, col[h], x);
        }
      }
    }
    if (++s == a.stages) {
      s = 0;
      phase ^= 1;
    }
  }
#pragma unroll
  for (int h = 0; h < kNormGradGroups; ++h) {
    if (live[h]) {
      const int64_t at = static_cast<int64_t>(part) * a.K + k0;
      if (a.part_a) store_pairs<T, true, 2>(a.part_a + at, col[h], acc_a[h]);
      if (a.part_b) store_pairs<T, true, 2>(a.part_b + at, col[h], acc_b[h]);
    }
  }
  if (*abort_flag) {  // copies in flight land before the CTA's memory goes
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 10000000ull) {
    }
  }
  if (a.slices > 1) cluster_meet();  // no CTA leaves while another writes its sums
}

// out[j, k] = sum over `count` partial rows of part[j * count + p, k], in a fixed order: a thread takes
// four columns and every 16th row, eight rows of loads in flight, and the 16 are added at the end.
// blockIdx.y: the output rows of all (at most three) sums, one after the other; a CTA that finds
// nothing to do still costs its launch, so none is made for them.
struct SumJob {
  const float *part;
  float *out;
  int rows;   // output rows
  int count;  // partial rows of each
};
struct SumJobs {
  SumJob job[3];
  int K;
};
constexpr int kSumCols = 16;  // threads of a CTA along K: 64 columns
constexpr int kSumRows = 16;  // along the partial rows
__global__ void __launch_bounds__(kSumCols *kSumRows) partial_sum_kernel(const SumJobs jobs) {
  __shared__ float4 red[kSumRows][kSumCols];
  pdl_wait();
  pdl_trigger();
  const int tx = threadIdx.x % kSumCols, ty = threadIdx.x / kSumCols;
  const int k = (static_cast<int>(blockIdx.x) * kSumCols + tx) * 4;
  const int total = jobs.job[0].rows + jobs.job[1].rows + jobs.job[2].rows;
  for (int at = blockIdx.y; at < total; at += gridDim.y) {
    int row = at, z = 0;
    while (row >= jobs.job[z].rows) row -= jobs.job[z++].rows;
    const SumJob j = jobs.job[z];
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (k < jobs.K) {
      const float *p = j.part + static_cast<int64_t>(row) * j.count * jobs.K + k;
#pragma unroll 8
      for (int i = ty; i < j.count; i += kSumRows) {
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(p + static_cast<int64_t>(i) * jobs.K));
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
      }
    }
    red[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && k < jobs.K) {
      for (int w = 1; w < kSumRows; ++w) {
        const float4 v = red[w][tx];
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
      }
      *reinterpret_cast<float4 *>(j.out + static_cast<int64_t>(row) * jobs.K + k) = s;
    }
    __syncthreads();
  }
}

template <class T, bool kR32, bool kOut8>
cudaError_t norm_forward(const NormArgs &a, int sms, cudaStream_t s) {
  const int chunks = a.K / 8;
  if (a.M <= 2 * sms) {  // few rows: as many threads as the row has chunks, straight from memory (latency)
    const int per = chunks <= 1024 ? 1 : 2;
    const dim3 grid(static_cast<unsigned>(a.M)), block(((chunks + per - 1) / per + 31) / 32 * 32);
    return per == 1 ? launch_pdl(residual_norm_kernel<T, kR32, 1, kOut8>, grid, block, 0, s, a)
                    : launch_pdl(residual_norm_kernel<T, kR32, 2, kOut8>, grid, block, 0, s, a);
  }
  // 16 columns per thread.  Up to 448 threads (K = 7168) two CTAs share an SM with 72 registers a
  // thread; more threads take one CTA per SM.
  const int threads = ((chunks + 1) / 2 + 31) / 32 * 32;
  const bool wide = threads > 448;
  const int stage = a.K * (2 + Res<T, kR32>::kBytes);
  int per_sm = wide ? 1 : 896 / threads;
  if (per_sm > 12) per_sm = 12;
  int stages = (kNormMaxSmem / per_sm - 2048) / stage;
  while (stages < 2 && per_sm > 1) stages = (kNormMaxSmem / --per_sm - 2048) / stage;
  if (stages > kNormMaxStages) stages = kNormMaxStages;
  if (stages < 1) stages = 1;
  const int smem = stages * stage;
  const int64_t cap = static_cast<int64_t>(sms) * per_sm;
  const dim3 grid(static_cast<unsigned>(a.M < cap ? a.M : cap)), block(threads);
  auto kernel = wide ? residual_norm_rows_kernel<T, kR32, 2, 1024, 1, kOut8> : residual_norm_rows_kernel<T, kR32, 2, 448, 2, kOut8>;
  static std::atomic<bool> ready[64][2];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev][wide].load()) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormMaxSmem);
    if (e != cudaSuccess) return e;
    ready[dev][wide].store(true);
  }
  return launch_pdl(kernel, grid, block, smem, s, a, stages);
}

template <class T, bool kR32>
cudaError_t norm_backward(const NormGradArgs &a, const NormGradPlan &p, cudaStream_t s) {
  auto kernel = residual_norm_backward_kernel<T, kR32>;
  static std::atomic<bool> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev].load()) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormMaxSmem);
    if (e != cudaSuccess) return e;
    ready[dev].store(true);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.ctas * p.slices));
  cfg.blockDim = dim3(p.threads);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.slices;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kernel, a);
  if (e != cudaSuccess) return e;
  SumJobs jobs = {};
  jobs.K = a.K;
  int n = 0, rows = 0;
  if (a.part_a) jobs.job[n++] = {a.part_a, a.dga, 1, p.ctas};
  if (a.part_b) jobs.job[n++] = {a.part_b, a.dgb, 1, p.ctas};
  if (a.part_g) {
    jobs.job[n++] = {a.part_g, a.dgate, static_cast<int>(a.groups), a.parts};
  }
  for (int i = 0; i < n; ++i) rows += jobs.job[i].rows;
  if (n == 0) return cudaSuccess;
  return launch_pdl(partial_sum_kernel, dim3((a.K + 4 * kSumCols - 1) / (4 * kSumCols), rows < 1024 ? rows : 1024),
                    dim3(kSumCols * kSumRows), 0, s, jobs);
}

}  // namespace

// How the backward spreads over the GPU (also decides the workspace, so it depends on sizes alone).
NormGradPlan norm_grad_plan(int64_t M, int64_t K, int64_t groups, bool r32) {
  NormGradPlan p;
  p.slices = static_cast<int>((K + kNormSlice - 1) / kNormSlice);
  p.slice_cols = static_cast<int>(((K + p.slices - 1) / p.slices + 7) / 8 * 8);
  p.threads = (p.slice_cols + 128 * kNormGradGroups - 1) / (128 * kNormGradGroups) * 32;
  const int stage = p.slice_cols * (r32 ? 12 : 8);
  // narrow rows: several CTAs per SM share its shared memory
  int per_sm = kNormGradThreads / p.threads;
  if (per_sm > kNormGradMaxCtas) per_sm = kNormGradMaxCtas;
  if (per_sm < 1) per_sm = 1;
  const int budget = (kNormMaxSmem - 1024) / per_sm - 1024;
  p.stages = budget / stage;
  if (p.stages > kNormMaxStages) p.stages = kNormMaxStages;
  if (p.stages < 1) p.stages = 1;
  p.smem = p.stages * stage;
  const int64_t want = static_cast<int64_t>(kNormSms) * per_sm / p.slices;
  const int64_t rows_per_group = groups > 0 ? M / groups : M;
  if (groups >= want) {
    p.parts = 1;
    p.ctas = static_cast<int>(want);
  } else {
    // few rows per CTA cost more in partial sums than they save: at least kNormGradRows each, as
    // long as every SM still has a CTA
    const int64_t base = kNormSms / p.slices;
    int64_t goal = M / kNormGradRows;
    if (goal < base) goal = base;
    if (goal > want) goal = want;
    int64_t parts = goal / (groups > 0 ? groups : 1);
    if (parts > rows_per_group) parts = rows_per_group;
    if (parts < 1) parts = 1;
    p.parts = static_cast<int>(parts);
    p.ctas = static_cast<int>(groups * parts);
  }
  return p;
}

template <class T>
static cudaError_t norm_as(const NormArgs &a, bool r32, int sms, cudaStream_t s) {
  if (a.q) return r32 ? norm_forward<T, true, true>(a, sms, s) : norm_forward<T, false, true>(a, sms, s);
  return r32 ? norm_forward<T, true, false>(a, sms, s) : norm_forward<T, false, false>(a, sms, s);
}
cudaError_t launch_residual_norm(const NormArgs &a, int dtype, bool r32, int sms, cudaStream_t s) {
  return dtype == NVFP4_DT_BF16 ? norm_as<Bf16>(a, r32, sms, s) : norm_as<Fp16>(a, r32, sms, s);
}

cudaError_t launch_residual_norm_backward(const NormGradArgs &a, const NormGradPlan &p, int dtype, bool r32,
                                          cudaStream_t s) {
  if (dtype == NVFP4_DT_BF16) return r32 ? norm_backward<Bf16, true>(a, p, s) : norm_backward<Bf16, false>(a, p, s);
  return r32 ? norm_backward<Fp16, true>(a, p, s) : norm_backward<Fp16, false>(a, p, s);
}

}  // namespace nvfp4
