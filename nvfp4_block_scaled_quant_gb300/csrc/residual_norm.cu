// The boundary between two blocks of a layer in one pass over memory:
//
//   n  = f rstd(f) ga          (the norm after the block; n = f without ga)
//   r' = r + scale gate n      (gate: one value per channel of a group of rows, or one per row)
//   y  = r' rstd(r') gb        (the norm before the next block; from r' before its rounding)
//
// with rstd(v) = 1 / sqrt(mean(v^2) + eps) over a row, all in fp32, and its backward pass.
//
// Backward of one row, with fh = f rstd(f), rh = r' rstd(r'), v = dy gb, and the sums over the row
//   c2 = sum v rh,  A = sum q (dr' + ib v),  C = sum q rh,  q = n gate (n alone for a gate per row):
//   dR    = dr' + ib (v - rh c2 / K)           the gradient of r' (and of r)
//   S     = sum q dR = A - ib c2 C / K
//   dgate = scale dR n                         (a gate per row: scale S)
//   df    = ia (scale gate dR ga - fh scale [gate] S / K)
//   dga  += scale gate dR fh,   dgb += dy rh
// S is linear in dR, so the three sums come from one sweep and one reduction over the block.
// rstd(f) and rstd(r') are kept by the forward (8 bytes per row); everything else is recomputed.
//
// Both passes are bound by memory: forward f + r in, r' + y out; backward f, r, dr', dy in, df, dr
// out.  Parameter gradients are held in fp32 registers over a CTA's rows (a thread keeps the same 8
// columns), written once per CTA and added in a fixed order by a second kernel: no atomics, so
// repeated calls give identical bits.
#include <atomic>

#include "mma16x8.cuh"

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

// The same four elements at a time.
template <class T, bool kF32>
struct Four {
  static __device__ __forceinline__ void load(const void *p, int64_t i, float (&v)[4]) {
    if constexpr (kF32) {
      const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    } else {
      const uint2 a = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i);
      v[0] = T::lo(a.x), v[1] = T::hi(a.x), v[2] = T::lo(a.y), v[3] = T::hi(a.y);
    }
  }
  static __device__ __forceinline__ void store(void *p, int64_t i, const float (&v)[4]) {
    if constexpr (kF32)
      *reinterpret_cast<float4 *>(static_cast<float *>(p) + i) = make_float4(v[0], v[1], v[2], v[3]);
    else
      *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p) + i) = make_uint2(T::pack(v[0], v[1]), T::pack(v[2], v[3]));
  }
};
// Element i of four packed 16-bit values.
template <class T>
__device__ __forceinline__ float at4(const uint2 w, int i) {
  const uint32_t x = i < 2 ? w.x : w.y;
  return (i & 1) ? T::hi(x) : T::lo(x);
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

__device__ __forceinline__ float rstd_of(float sum, int K, float eps) {
  return __fdiv_rn(1.f, __fsqrt_rn(__fdiv_rn(sum, static_cast<float>(K)) + eps));
}

// ---------------------------------------------------------------- forward

// Few rows: one row per CTA, kChunks groups of 8 columns per thread, in registers over both
// reductions.
template <class T, bool kR32, int kChunks>
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
      ia = rstd_of(block_sum(s, red[0]), a.K, a.eps);
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
      ib = rstd_of(block_sum(s, red[1]), a.K, a.eps);
#pragma unroll
      for (int u = 0; u < kChunks; ++u) {
        const int c = static_cast<int>(threadIdx.x) + u * nt;
        if (c < chunks) {
          float gb[8], y[8];
          load_opt<T>(static_cast<const uint16_t *>(a.gb), c * 8, 1.f, gb);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = rv[u][i] * ib * gb[i];
          Res<T, false>::store(a.y, m * a.K + c * 8, y);
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
template <class T, bool kR32, int kChunks>
__global__ void __launch_bounds__(1024, 1) residual_norm_rows_kernel(const NormArgs a, int stages) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) &
                                              ~static_cast<uintptr_t>(127));
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
  float next_gm = a.gate_kind == NVFP4_GATE_ROW && blockIdx.x < a.M ? T::up(__ldg(gate0 + blockIdx.x)) : 1.f;
  for (int64_t m = blockIdx.x; m < a.M; m += step) {
    const float gm = a.scale * next_gm;
    if (a.gate_kind == NVFP4_GATE_ROW && m + step < a.M) next_gm = T::up(__ldg(gate0 + m + step));
    const uint16_t *gate = a.gate_kind == NVFP4_GATE_CHANNEL ? gate0 + static_cast<int64_t>(group_of(m, a.rows_per_group)) * a.K : nullptr;
    // a wait that gives up raises the fault flag; every barrier below is still met
    mbar_wait_bounded(&full[s], phase, abort_flag, a.err, kPipelineTimeoutNs);
    const uint8_t *d = smem + s * stage_bytes;
    float v[kChunks][8];
    float sum = 0.f;
    float ia = 1.f;
    if (a.ga) {
#pragma unroll
      for (int u = 0; u < kChunks; ++u) {
        const int c = tid + u * nt;
        if (c < chunks) {
          Res<T, false>::load(d, c * 8, v[u]);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum += v[u][i] * v[u][i];
        }
      }
      ia = rstd_of(block_sum(sum, red[0]), a.K, a.eps);
    }
    sum = 0.f;
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
      const int c = tid + u * nt;
      if (c < chunks) {
        float x[8], w[8];
        if (!a.ga) Res<T, false>::load(d, c * 8, v[u]);
        load_opt<T>(static_cast<const uint16_t *>(a.ga), c * 8, 1.f, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] *= ia * w[i];
        load_opt<T>(gate, c * 8, 1.f, w);
        Res<T, kR32>::load(d + n16, c * 8, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[u][i] = x[i] + gm * w[i] * v[u][i];
          sum += v[u][i] * v[u][i];
        }
        Res<T, kR32>::store(a.r_out, m * a.ldr_out + c * 8, v[u]);
      }
    }
    float ib = 0.f;
    if (a.gb) {
      ib = rstd_of(block_sum(sum, red[1]), a.K, a.eps);  // its barrier: every thread has read the stage
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
          float gb[8];
          load_opt<T>(static_cast<const uint16_t *>(a.gb), c * 8, 1.f, gb);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[u][i] *= ib * gb[i];
          Res<T, false>::store(a.y, m * a.K + c * 8, v[u]);
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
// load while this one is reduced; registers hold the parameter gradients.  A row of more than
// kNormSlice columns is split over the CTAs of a cluster, which exchange the three sums.
constexpr int kNbRedFloats = 4 * 32;  // three sums of up to 32 warps each, and a row of zeros

template <class T, bool kR32>
__global__ void __launch_bounds__(kNormGradThreads, 1) residual_norm_backward_kernel(const NormGradArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) &
                                              ~static_cast<uintptr_t>(127));
  __shared__ __align__(16) float red[2][kNbRedFloats];
  __shared__ float peer_sums[2][kNormMaxSlices][3];
  __shared__ uint64_t full[kNormMaxStages];
  __shared__ int s_abort;
  volatile int *abort_flag = &s_abort;

  const int slice = static_cast<int>(blockIdx.x) % a.slices, part = static_cast<int>(blockIdx.x) / a.slices;
  const int k0 = slice * a.slice_cols, cols = min(a.slice_cols, a.K - k0);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // this thread's columns of the slice: two groups of four, each contiguous over the block
  const int col[2] = {static_cast<int>(threadIdx.x) * 4, static_cast<int>(blockDim.x + threadIdx.x) * 4};
  const bool live[2] = {col[0] < cols, col[1] < cols};
  // ring stage: f, dy (16 bits), r, dr' (16 or 32 bits), each slice_cols wide
  const int b16 = a.slice_cols * 2, br = a.slice_cols * Res<T, kR32>::kBytes;
  const int stage_bytes = 2 * b16 + 2 * br;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) mbar_init(&full[s], 1);
    s_abort = 0;
    fence_barrier_init();
  }
  for (int i = static_cast<int>(threadIdx.x); i < 2 * kNbRedFloats; i += static_cast<int>(blockDim.x)) red[0][i] = 0.f;
  __syncthreads();
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
  auto load_row = [&](int64_t m) {
    const int s = static_cast<int>((m - m_first) % a.stages);
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
    for (int64_t m = m_first; m < m_last && m < m_first + a.stages; ++m) load_row(m);

  const uint16_t *gp = static_cast<const uint16_t *>(a.gate);
  const bool row_gate = a.gate_kind == NVFP4_GATE_ROW, channel_gate = a.gate_kind == NVFP4_GATE_CHANNEL;
  const float inv_k = 1.f / static_cast<float>(a.K);
  // parameters of the thread's columns, packed as stored; the gate's change with the group of rows
  uint2 ga[2], gb[2], gk[2];
  const uint32_t one = T::pack(1.f, 1.f);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    ga[h] = gk[h] = make_uint2(one, one);
    gb[h] = make_uint2(0u, 0u);
    if (live[h]) {
      if (a.ga) ga[h] = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.ga) + k0 + col[h]));
      if (a.gb) gb[h] = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.gb) + k0 + col[h]));
    }
  }
  float acc_a[2][4], acc_b[2][4], acc_g[2][4];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc_a[h][i] = acc_b[h][i] = acc_g[h][i] = 0.f;

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
      if (channel_gate) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (live[h]) gk[h] = __ldg(reinterpret_cast<const uint2 *>(gp + group * a.K + k0 + col[h]));
      }
    }
    --rows_left;
    // a wait that gives up leaves this CTA's results undefined and the fault flag raised, but every
    // barrier below is still met
    mbar_wait_bounded(&full[s], phase, abort_flag, a.err, kPipelineTimeoutNs);
    const uint8_t *d = smem + s * stage_bytes;
    float fv[4], rv[4], dyv[4], drv[4], w[4];
    auto fetch = [&](int h) {
      Four<T, false>::load(d, col[h], fv);
      Four<T, kR32>::load(d + 2 * b16, col[h], rv);
#pragma unroll
      for (int i = 0; i < 4; ++i) dyv[i] = drv[i] = 0.f;
      if (a.dy) Four<T, false>::load(d + b16, col[h], dyv);
      if (a.dr_out) Four<T, kR32>::load(d + 2 * b16 + br, col[h], drv);
    };
    float c2 = 0.f, sa = 0.f, sc = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (live[h]) {
        fetch(h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float q = at4<T>(gk[h], i) * (fv[i] * ia * at4<T>(ga[h], i));
          const float rh = (rv[i] + gm * q) * ib, v = dyv[i] * at4<T>(gb[h], i);
          c2 += v * rh;
          sa += q * (drv[i] + ib * v);
          sc += q * rh;
        }
      }
    }
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
    __syncthreads();  // also: every thread is done with the previous row's stage
    if (threadIdx.x == 0 && m > m_first && m - 1 + a.stages < m_last) load_row(m - 1 + a.stages);
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
      __syncwarp();
      cluster_sync();
      c2 = sa = sc = 0.f;
      for (int r = 0; r < a.slices; ++r) {
        c2 += peer_sums[pb][r][0];
        sa += peer_sums[pb][r][1];
        sc += peer_sums[pb][r][2];
      }
    }
    const float mean2 = c2 * inv_k;
    const float S = sa - ib * mean2 * sc;  // sum q dR
    const float mean1 = gm * S * inv_k;    // mean of fh times the gradient of fh
    if (row_gate && a.dgate && threadIdx.x == 0 && slice == 0) a.dgate[m] = a.scale * S;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (live[h]) {
        fetch(h);
        float df[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float fh = fv[i] * ia, g = at4<T>(ga[h], i), k = at4<T>(gk[h], i), n = fh * g;
          const float rh = (rv[i] + gm * k * n) * ib, v = dyv[i] * at4<T>(gb[h], i);
          acc_b[h][i] += dyv[i] * rh;
          w[i] = drv[i] + ib * (v - rh * mean2);
          const float sdr = gm * w[i];
          acc_g[h][i] += sdr * n;
          const float dn = sdr * k;
          acc_a[h][i] += dn * fh;
          df[i] = a.ga ? ia * (dn * g - fh * mean1) : dn;
        }
        Four<T, kR32>::store(a.dr, m * a.K + k0 + col[h], w);
        Four<T, false>::store(a.df, m * a.K + k0 + col[h], df);
      }
    }
    if (rows_left == 0 && channel_gate && a.dgate) {  // the end of a group of rows: its gate gradient
      const int64_t at = (a.parts > 1 ? part : group) * a.K + k0;
      float *dst = (a.parts > 1 ? a.part_g : a.dgate) + at;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (live[h]) Four<T, true>::store(dst, col[h], acc_g[h]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc_g[h][i] = 0.f;
      }
    }
    if (++s == a.stages) {
      s = 0;
      phase ^= 1;
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (live[h]) {
      const int64_t at = static_cast<int64_t>(part) * a.K + k0;
      if (a.part_a) Four<T, true>::store(a.part_a + at, col[h], acc_a[h]);
      if (a.part_b) Four<T, true>::store(a.part_b + at, col[h], acc_b[h]);
    }
  }
  if (*abort_flag) {  // copies in flight land before the CTA's memory goes
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 10000000ull) {
    }
  }
  if (a.slices > 1) cluster_sync();  // no CTA leaves while another writes its sums
}

// out[j, k] = sum over `count` partial rows of part[j * count + p, k], in a fixed order: a warp's 32
// lanes take 32 columns, the 8 warps of a CTA every eighth row.  blockIdx.y: the output row j;
// blockIdx.z: which of the (at most three) sums.
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
__global__ void __launch_bounds__(256) partial_sum_kernel(const SumJobs jobs) {
  __shared__ float red[8][32];
  pdl_wait();
  pdl_trigger();
  const SumJob j = jobs.job[blockIdx.z];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, k = static_cast<int>(blockIdx.x) * 32 + lane;
  for (int row = blockIdx.y; row < j.rows; row += gridDim.y) {
    float s = 0.f;
    if (k < jobs.K) {
      const float *p = j.part + static_cast<int64_t>(row) * j.count * jobs.K + k;
#pragma unroll 4
      for (int i = warp; i < j.count; i += 8) s += __ldg(p + static_cast<int64_t>(i) * jobs.K);
    }
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && k < jobs.K) {
      s = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) s += red[w][lane];
      j.out[static_cast<int64_t>(row) * jobs.K + k] = s;
    }
    __syncthreads();
  }
}

template <class T, bool kR32>
cudaError_t norm_forward(const NormArgs &a, int sms, cudaStream_t s) {
  const int chunks = a.K / 8;
  if (a.M <= 2 * sms) {  // few rows: as many threads as the row has chunks, straight from memory (latency)
    const int per = chunks <= 1024 ? 1 : 2;
    const dim3 grid(static_cast<unsigned>(a.M)), block(((chunks + per - 1) / per + 31) / 32 * 32);
    return per == 1 ? launch_pdl(residual_norm_kernel<T, kR32, 1>, grid, block, 0, s, a)
                    : launch_pdl(residual_norm_kernel<T, kR32, 2>, grid, block, 0, s, a);
  }
  const int per = chunks <= 64 ? 1 : 2;
  const int threads = ((chunks + per - 1) / per + 31) / 32 * 32;
  const int stage = a.K * (2 + Res<T, kR32>::kBytes);
  int per_sm = 1024 / threads;
  if (per_sm > 16) per_sm = 16;
  int stages = (kNormMaxSmem / per_sm - 2048) / stage;
  while (stages < 2 && per_sm > 1) stages = (kNormMaxSmem / --per_sm - 2048) / stage;
  if (stages > kNormMaxStages) stages = kNormMaxStages;
  if (stages < 1) stages = 1;
  const int smem = 128 + stages * stage;
  const int64_t cap = static_cast<int64_t>(sms) * per_sm;
  const dim3 grid(static_cast<unsigned>(a.M < cap ? a.M : cap)), block(threads);
  auto kernel = per == 1 ? residual_norm_rows_kernel<T, kR32, 1> : residual_norm_rows_kernel<T, kR32, 2>;
  static std::atomic<bool> ready[64][2];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev][per - 1].load()) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormMaxSmem);
    if (e != cudaSuccess) return e;
    ready[dev][per - 1].store(true);
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
  int n = 0, rows = 1;
  if (a.part_a) jobs.job[n++] = {a.part_a, a.dga, 1, p.ctas};
  if (a.part_b) jobs.job[n++] = {a.part_b, a.dgb, 1, p.ctas};
  if (a.part_g) {
    jobs.job[n++] = {a.part_g, a.dgate, static_cast<int>(a.groups), a.parts};
    rows = static_cast<int>(a.groups);
  }
  if (n == 0) return cudaSuccess;
  return launch_pdl(partial_sum_kernel, dim3((a.K + 31) / 32, rows < 1024 ? rows : 1024, n), dim3(256), 0, s, jobs);
}

}  // namespace

// How the backward spreads over the GPU (also decides the workspace, so it depends on sizes alone).
NormGradPlan norm_grad_plan(int64_t M, int64_t K, int64_t groups, bool r32) {
  NormGradPlan p;
  p.slices = static_cast<int>((K + kNormSlice - 1) / kNormSlice);
  p.slice_cols = static_cast<int>(((K + p.slices - 1) / p.slices + 7) / 8 * 8);
  p.threads = (p.slice_cols / 8 + 31) / 32 * 32;
  const int stage = p.slice_cols * (r32 ? 12 : 8);
  // narrow rows: several CTAs per SM share its shared memory
  int per_sm = kNormGradThreads / p.threads;
  if (per_sm > 8) per_sm = 8;
  if (per_sm < 1) per_sm = 1;
  const int budget = (kNormMaxSmem - 1024) / per_sm - 1024;
  p.stages = budget / stage;
  if (p.stages > kNormMaxStages) p.stages = kNormMaxStages;
  if (p.stages < 1) p.stages = 1;
  p.smem = 128 + p.stages * stage;
  const int64_t want = static_cast<int64_t>(kNormSms) * per_sm / p.slices;
  const int64_t rows_per_group = groups > 0 ? M / groups : M;
  if (groups >= want) {
    p.parts = 1;
    p.ctas = static_cast<int>(want);
  } else {
    int64_t parts = want / (groups > 0 ? groups : 1);
    if (parts > rows_per_group) parts = rows_per_group;
    if (parts < 1) parts = 1;
    p.parts = static_cast<int>(parts);
    p.ctas = static_cast<int>(groups * parts);
  }
  return p;
}

cudaError_t launch_residual_norm(const NormArgs &a, int dtype, bool r32, int sms, cudaStream_t s) {
  if (dtype == NVFP4_DT_BF16) return r32 ? norm_forward<Bf16, true>(a, sms, s) : norm_forward<Bf16, false>(a, sms, s);
  return r32 ? norm_forward<Fp16, true>(a, sms, s) : norm_forward<Fp16, false>(a, sms, s);
}

cudaError_t launch_residual_norm_backward(const NormGradArgs &a, const NormGradPlan &p, int dtype, bool r32,
                                          cudaStream_t s) {
  if (dtype == NVFP4_DT_BF16) return r32 ? norm_backward<Bf16, true>(a, p, s) : norm_backward<Bf16, false>(a, p, s);
  return r32 ? norm_backward<Fp16, true>(a, p, s) : norm_backward<Fp16, false>(a, p, s);
}

}  // namespace nvfp4
