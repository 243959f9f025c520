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

__device__ __forceinline__ float rstd_of(float sum, int K, float eps) {
  return __fdiv_rn(1.f, __fsqrt_rn(__fdiv_rn(sum, static_cast<float>(K)) + eps));
}

// ---------------------------------------------------------------- forward

// A row per CTA at a time; kChunks groups of 8 columns per thread stay in registers over both
// reductions, so memory is read once.
template <class T, bool kR32, int kChunks>
__global__ void __launch_bounds__(kChunks == 4 ? 512 : 1024, 1) residual_norm_kernel(const NormArgs a) {
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
      gate += m / a.rows_per_group * a.K;
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

// ---------------------------------------------------------------- backward

// Rows stream through a ring in shared memory (one bulk copy per row and tensor), so the next rows
// load while this one is reduced; registers hold the parameter gradients.  A row of more than
// kNormSlice columns is split over the CTAs of a cluster, which exchange the three sums.
constexpr int kNbRedFloats = 3 * 32;

template <class T, bool kR32>
__global__ void __launch_bounds__(1024, 1) residual_norm_backward_kernel(const NormGradArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) &
                                              ~static_cast<uintptr_t>(127));
  __shared__ float red[2][kNbRedFloats];
  __shared__ float peer_sums[2][kNormMaxSlices][3];
  __shared__ uint64_t full[kNormMaxStages];
  __shared__ int s_abort;
  volatile int *abort_flag = &s_abort;

  const int slice = static_cast<int>(blockIdx.x) % a.slices, part = static_cast<int>(blockIdx.x) / a.slices;
  const int k0 = slice * a.slice_cols, cols = min(a.slice_cols, a.K - k0);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = static_cast<int>(blockDim.x) >> 5;
  const int c = static_cast<int>(threadIdx.x) * 8;  // this thread's columns of the slice
  const bool live = c < cols;
  // ring stage: f, dy (16 bits), r, dr' (16 or 32 bits), each slice_cols wide
  const int b16 = a.slice_cols * 2, br = a.slice_cols * Res<T, kR32>::kBytes;
  const int stage_bytes = 2 * b16 + 2 * br;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) mbar_init(&full[s], 1);
    s_abort = 0;
    fence_barrier_init();
  }
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
  const float inv_k = 1.f / static_cast<float>(a.K);
  float acc_a[8], acc_b[8], acc_g[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc_a[i] = acc_b[i] = acc_g[i] = 0.f;

  for (int64_t m = m_first; m < m_last; ++m) {
    const int64_t i_row = m - m_first;
    const int s = static_cast<int>(i_row % a.stages);
    const int pb = static_cast<int>(i_row & 1);
    // a wait that gives up leaves this CTA's results undefined and the fault flag raised, but every
    // barrier below is still met
    mbar_wait_bounded(&full[s], static_cast<uint32_t>(i_row / a.stages) & 1u, abort_flag, a.err, kPipelineTimeoutNs);
    const uint8_t *d = smem + s * stage_bytes;
    const float2 st = __ldg(reinterpret_cast<const float2 *>(a.stats) + m);
    const float ia = a.ga ? st.x : 1.f, ib = st.y;
    float gm = a.scale;
    const uint16_t *gate = gp;
    if (a.gate_kind == NVFP4_GATE_ROW) {
      gm *= T::up(__ldg(gp + m));
      gate = nullptr;
    } else if (gp) {
      gate += m / a.rows_per_group * a.K + k0;
    }

    // one column: q, rh, v and dr' (fh = f ia and n = fh ga are recomputed where needed)
    float fv[8], rv[8], dyv[8], drv[8], ga[8], gb[8], gk[8];
    float c2 = 0.f, sa = 0.f, sc = 0.f;
    auto fetch = [&]() {
      Res<T, false>::load(d, c, fv);
      Res<T, kR32>::load(d + 2 * b16, c, rv);
#pragma unroll
      for (int i = 0; i < 8; ++i) dyv[i] = drv[i] = 0.f;
      if (a.dy) Res<T, false>::load(d + b16, c, dyv);
      if (a.dr_out) Res<T, kR32>::load(d + 2 * b16 + br, c, drv);
      load_opt<T>(a.ga ? static_cast<const uint16_t *>(a.ga) + k0 : nullptr, c, 1.f, ga);
      load_opt<T>(a.gb ? static_cast<const uint16_t *>(a.gb) + k0 : nullptr, c, 0.f, gb);
      load_opt<T>(gate, c, 1.f, gk);
    };
    if (live) {
      fetch();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float q = gk[i] * (fv[i] * ia * ga[i]);
        const float rh = (rv[i] + gm * q) * ib, v = dyv[i] * gb[i];
        c2 += v * rh;
        sa += q * (drv[i] + ib * v);
        sc += q * rh;
      }
    }
    c2 = warp_sum(c2);
    sa = warp_sum(sa);
    sc = warp_sum(sc);
    if (lane == 0) {
      red[pb][warp] = c2;
      red[pb][32 + warp] = sa;
      red[pb][64 + warp] = sc;
    }
    __syncthreads();  // also: every thread is done with the previous row's stage
    if (threadIdx.x == 0 && i_row > 0 && m - 1 + a.stages < m_last) load_row(m - 1 + a.stages);
    c2 = warp_sum(lane < warps ? red[pb][lane] : 0.f);
    sa = warp_sum(lane < warps ? red[pb][32 + lane] : 0.f);
    sc = warp_sum(lane < warps ? red[pb][64 + lane] : 0.f);
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
    const float S = sa - ib * mean2 * sc;                // sum q dR
    const float mean1 = gm * S * inv_k;                  // mean of fh times the gradient of fh
    if (a.gate_kind == NVFP4_GATE_ROW && a.dgate && threadIdx.x == 0 && slice == 0) a.dgate[m] = a.scale * S;
    if (live) {
      fetch();
      float dr[8], df[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float fh = fv[i] * ia, n = fh * ga[i];
        const float rh = (rv[i] + gm * gk[i] * n) * ib, v = dyv[i] * gb[i];
        dr[i] = drv[i] + ib * (v - rh * mean2);
        const float sdr = gm * dr[i];
        acc_b[i] += dyv[i] * rh;
        acc_g[i] += sdr * n;
        const float dn = sdr * gk[i];
        acc_a[i] += dn * fh;
        df[i] = a.ga ? ia * (dn * ga[i] - fh * mean1) : dn;
      }
      Res<T, kR32>::store(a.dr, m * a.K + k0 + c, dr);
      Res<T, false>::store(a.df, m * a.K + k0 + c, df);
      // the end of a group of rows: its gate gradient
      if (a.gate_kind == NVFP4_GATE_CHANNEL && a.dgate && (m + 1 == m_last || (m + 1) % a.rows_per_group == 0)) {
        const int64_t at = (a.parts > 1 ? part : m / a.rows_per_group) * a.K + k0 + c;
        float *dst = (a.parts > 1 ? a.part_g : a.dgate) + at;
        reinterpret_cast<float4 *>(dst)[0] = make_float4(acc_g[0], acc_g[1], acc_g[2], acc_g[3]);
        reinterpret_cast<float4 *>(dst)[1] = make_float4(acc_g[4], acc_g[5], acc_g[6], acc_g[7]);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc_g[i] = 0.f;
      }
    }
  }
  if (live) {
    const int64_t at = static_cast<int64_t>(part) * a.K + k0 + c;
    if (a.part_a) {
      reinterpret_cast<float4 *>(a.part_a + at)[0] = make_float4(acc_a[0], acc_a[1], acc_a[2], acc_a[3]);
      reinterpret_cast<float4 *>(a.part_a + at)[1] = make_float4(acc_a[4], acc_a[5], acc_a[6], acc_a[7]);
    }
    if (a.part_b) {
      reinterpret_cast<float4 *>(a.part_b + at)[0] = make_float4(acc_b[0], acc_b[1], acc_b[2], acc_b[3]);
      reinterpret_cast<float4 *>(a.part_b + at)[1] = make_float4(acc_b[4], acc_b[5], acc_b[6], acc_b[7]);
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
  // few rows: as many threads as the row has chunks (latency); many rows: four chunks per thread,
  // more CTAs per SM and more loads in flight per thread
  const int per = a.M <= 2 * sms ? (chunks <= 1024 ? 1 : 2) : (chunks <= 128 ? 1 : chunks <= 512 ? 2 : 4);
  const int threads = ((chunks + per - 1) / per + 31) / 32 * 32;
  const int64_t cap = static_cast<int64_t>(sms) * 16;
  const dim3 grid(static_cast<unsigned>(a.M < cap ? a.M : cap)), block(threads);
  switch (per) {
    case 1: return launch_pdl(residual_norm_kernel<T, kR32, 1>, grid, block, 0, s, a);
    case 2: return launch_pdl(residual_norm_kernel<T, kR32, 2>, grid, block, 0, s, a);
  }
  return launch_pdl(residual_norm_kernel<T, kR32, 4>, grid, block, 0, s, a);
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
  int per_sm = 1024 / p.threads;
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
