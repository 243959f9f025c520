// The linear layer on 4-bit weights for some ten to some hundred tokens, on the 5th-generation tensor cores in one launch.
//
// 128 weight rows (two prepared panels) are the MMA's M and kTok tokens its N; the reduction is split over the CTAs of a
// cluster so that every SM takes part where there are few tiles, and their sums are added through distributed shared
// memory in rank order.  Codes stream into a ring of their own, 128 K of both panels by two bulk copies; dequantising
// warps write (c - z) 2^-e, exact in either type, into 64-wide stages of the MMA's A operand, beside which TMA puts the
// tokens.  Each group's product goes to an accumulator of its own, and the epilogue warps add it to fp32 registers
// times the scale of their row, which they read from the ring: no weight is rounded.
//
// What a stage takes in turn (codes, dequantisation, commit, promotion) bounds it: 64 rows 7168 -> 7168 22.3 us (1.2 TB/s of
// weights), 128 rows 27.7 (475 TF/s).
// Warps: 0 = codes, 1 and 3 = MMA (3 also tensor memory), 2 = tokens, then the epilogue (four warps for each 64 tokens, one
// 32-row quarter of tensor memory each) and the dequantising warps.  Every wait is bounded, as in the other
// kernels; what hangs on the tokens waits for the previous launch first, whose time does not count.
#include "w4.cuh"

namespace nvfp4 {
namespace {

template <int kGpb, bool kZeros, int kTok>
struct TcCfg {
  static constexpr int kBlock = w4_block_bytes(kGpb, kZeros);
  static constexpr int kABytes = 128 * 128;                     // 128 rows x 64 K
  static constexpr int kXBytes = kTok * 128;
  static constexpr int kStages = 4;                             // of A
  // tokens arrive from L2 in about a microsecond, in which several stages pass: a longer ring of their own
  static constexpr int kXStages = kTok > 64 ? 6 : kTok > 32 ? 8 : 16;
  static constexpr int kCodes = kTok > 64 ? 6 : 8;              // 128 K of both panels each
  static constexpr int kRing = kStages * kABytes + kXStages * kXBytes;
  // Accumulators.  The epilogue follows the stages' barriers, so the MMAs may not get four stages ahead of it: two for
  // groups of two stages.  Each belongs to one issuer: four where a stage holds two groups.
  static constexpr int kBufs = kGpb == 1 ? 2 : kGpb == 4 || kTok <= 64 ? 4 : 2;
  static constexpr uint32_t kTmemCols = kBufs * kTok;
  static constexpr int kEpi = kTok > 64 ? 8 : 4, kDeq = 12 - kEpi;
  static constexpr int kThreads = 512;
  static constexpr size_t kSmem = kRing + kCodes * 2 * kBlock + 1024;
  static_assert(kSmem <= 232448 - 1024, "per-block shared memory limit");
  static_assert(kTok * 128 * 4 <= kRing, "the sums fit where the ring was");
  static_assert(kDeq % kStages == 0 && kCodes % 2 == 0, "a warp sees every phase of the barriers it waits on");
  static_assert(kTok % 32 == 0 && kTmemCols <= 512, "MMA N, tensor memory");
  // The issuer of a 64-wide step (they take the groups of 128, else the steps, in turn), and its tokens' stage: each issuer has
  // half of the ring, of which it sees every phase.
  static __device__ __forceinline__ int issuer(int step) { return kGpb == 1 ? (step >> 1) & 1 : step & 1; }
  static __device__ __forceinline__ int turn(int step) { return kGpb == 1 ? (step >> 2) * 2 + (step & 1) : step >> 1; }
  static __device__ __forceinline__ int x_stage(int step) { return issuer(step) * (kXStages / 2) + turn(step) % (kXStages / 2); }
  static __device__ __forceinline__ uint32_t x_phase(int step) { return turn(step) / (kXStages / 2) & 1; }
};

template <class T, int kGpb, bool kZeros, int kTok>
__global__ void __launch_bounds__(512, 1) w4_tc_kernel(const __grid_constant__ CUtensorMap tmX, const W4Args args, const int splits) {
  using C = TcCfg<kGpb, kZeros, kTok>;
  constexpr uint32_t kIdesc = mma_idesc(T::kCode == NVFP4_DT_BF16 ? 1u : 0u, false, false, 128, kTok);
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *sA = smem, *sX = sA + C::kStages * C::kABytes, *sC = smem + C::kRing;
  __shared__ uint64_t full[C::kStages], done[C::kStages], full_x[C::kXStages], empty_x[C::kXStages], full_c[C::kCodes], empty_c[C::kCodes], tempty[C::kBufs];
  __shared__ uint32_t tmem_holder;
  __shared__ int s_abort;
  volatile int *abort_flag = &s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(blockIdx.x) % splits, tile = static_cast<int>(blockIdx.x) / splits;
  const int m0 = static_cast<int>(blockIdx.y) * kTok;
  const int blocks = (args.K + kW4BlockK - 1) / kW4BlockK, panels = (args.N + kW4PanelRows - 1) / kW4PanelRows;
  const int kb0 = static_cast<int>(static_cast<int64_t>(blocks) * rank / splits);
  const int kb1 = static_cast<int>(static_cast<int64_t>(blocks) * (rank + 1) / splits);
  const int mine = min(2, panels - 2 * tile);  // panels of the tile that exist

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], C::kDeq / C::kStages);
      mbar_init(&done[s], 1);
    }
    for (int s = 0; s < C::kXStages; ++s) {
      mbar_init(&full_x[s], 1);
      mbar_init(&empty_x[s], C::kDeq / C::kStages);
    }
    for (int s = 0; s < C::kCodes; ++s) {
      mbar_init(&full_c[s], 1);
      mbar_init(&empty_c[s], 2 * (C::kDeq / C::kStages) + C::kEpi);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      mbar_init(&tempty[b], C::kEpi);
    }
    s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 2 && lane == 0) prefetch_tensormap(&tmX);
  __syncwarp();
  if (warp == 3) {
    tmem_alloc(&tmem_holder, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  block_meet();
  tc_fence_after();
  const uint32_t tmem_base = tmem_holder;
  auto settle = [] {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 10000000ull) {
    }
  };
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    const bool ok = mbar_wait_bounded(bar, parity, abort_flag, args.err, kPipelineTimeoutNs);
    return __all_sync(0xffffffffu, ok) != 0;
  };
  bool ok = true;

  if (warp == 0) {
    // -------------------------------------------------------------- codes: prepared weights are final one launch early
    const uint64_t pol = policy_evict_normal();
    const uint8_t *w = args.w + static_cast<int64_t>(2 * tile) * blocks * C::kBlock;
    int stage = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (kb == kb0 + C::kCodes) pdl_wait();  // the ring is full: the next place hangs on the tokens
      ok = wait(&empty_c[stage], phase ^ 1);
      if (!ok) break;
      if (lane == 0) {
        uint8_t *dst = sC + stage * 2 * C::kBlock;
        mbar_arrive_expect_tx(&full_c[stage], mine * C::kBlock);
        for (int p = 0; p < mine; ++p)
          bulk_load(dst + p * C::kBlock, w + (static_cast<int64_t>(p) * blocks + kb) * C::kBlock, C::kBlock, &full_c[stage], pol);
      }
      __syncwarp();
      if (++stage == C::kCodes) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (!ok) settle();
  } else if (warp == 2) {
    // -------------------------------------------------------------- tokens
    pdl_wait();
    pdl_trigger();
    const uint64_t pol = policy_evict_last();
    for (int s = 0; s < 2 * (kb1 - kb0); ++s) {
      const int stage = C::x_stage(s);
      ok = wait(&empty_x[stage], C::x_phase(s) ^ 1);
      if (!ok) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(&full_x[stage], C::kXBytes);
        tma_load_2d(sX + stage * C::kXBytes, &tmX, (2 * kb0 + s) * 128, m0, &full_x[stage], pol);
      }
      __syncwarp();
    }
    if (!ok) settle();
  } else if (warp < 4) {
    // -------------------------------------------------------------- MMA issuers (one elected lane issues)
    // A commit takes its issuer some 200 cycles, waits and the rest of a stage about as much: one commit per stage, whose barrier everyone
    // follows (with one for the stage, one for the tokens and one for the accumulator, and one issuer, a tile of 16 tokens
    // 7168 -> 7168 took 30 us instead of 20), and two issuers that take the groups (of 32: the stages) in turn.
    pdl_wait();
    const int iss = warp >> 1;  // warps 1 and 3
    const uint32_t a0 = smem_u32(sA), x0 = smem_u32(sX);
    constexpr int kSteps = kGpb == 4 ? 2 : 4;       // MMAs of a group in a stage
    constexpr int kParts = 4 / kSteps;              // groups of a stage
    constexpr int kSpan = kGpb == 1 ? 2 : 1;        // stages of a turn
    const int steps = 2 * (kb1 - kb0);
    for (int s0 = iss * kSpan; ok && s0 < steps; s0 += 2 * kSpan) {
#pragma unroll
      for (int h = 0; h < kSpan; ++h) {
        const int s = s0 + h, stage = s % C::kStages, xs = C::x_stage(s);
        ok = wait(&full_x[xs], C::x_phase(s)) && wait(&full[stage], s / C::kStages & 1);
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
          const int n = kGpb == 1 ? s >> 1 : s * kParts + part, buf = n % C::kBufs;
          if (h == 0) ok = ok && wait(&tempty[buf], (n / C::kBufs & 1) ^ 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t ad = smem_desc(a0 + stage * C::kABytes, 16, 1024, 2), xd = smem_desc(x0 + xs * C::kXBytes, 16, 1024, 2);
#pragma unroll
            for (int j = 0; j < kSteps; ++j)
              tc_mma<false, false>(tmem_base + buf * kTok, ad + 2 * (part * kSteps + j), xd + 2 * (part * kSteps + j), kIdesc, (h | j) != 0);
            if (part == kParts - 1) tc_commit(&done[stage]);
          }
          __syncwarp();
        }
        if (!ok) break;
      }
    }
    if (!ok) settle();
  } else if (warp >= 4 + C::kEpi) {
    // -------------------------------------------------------------- dequantising warps
    // Each warp writes one stage of the ring, all of it or (kDeq = 8) one of its panels, so that four stages are in work at
    // once and a warp's steps (read, unpack, write, fence) overlap other warps'.  A unit is eight rows of four row tiles by
    // 64 K: row tile pair `pair`, rows g of one half of eight.  A quarter of the warp reads 4 t x 2 chunks of one
    // row, so that its 16-byte stores meet eight different banks under the swizzle.
    constexpr int kShare = C::kDeq / C::kStages, kUnits = 8 / kShare;
    const int w = warp - 4 - C::kEpi, stage = w % C::kStages, unit0 = w / C::kStages * kUnits;
    const int t = lane & 3, cb = (lane >> 2) & 1, steps = 2 * (kb1 - kb0);
    for (int s = stage; s < steps; s += C::kStages) {
      const int cs = (s >> 1) % C::kCodes;
      ok = wait(&full_c[cs], (s >> 1) / C::kCodes & 1);
      if (s >= C::kStages) {  // the stage's last product, which also was its tokens' last use
        if (s < 2 * C::kStages) pdl_wait();  // the warp's first stage was written meanwhile
        ok = ok && wait(&done[stage], (s / C::kStages & 1) ^ 1);
        if (ok && lane == 0) mbar_arrive(&empty_x[C::x_stage(s - C::kStages)]);
      }
      if (!ok) break;
      const int c = 2 * (s & 1) + cb, gi = c * kGpb / 4;
      uint4 v[kUnits];
#pragma unroll
      for (int q = 0; q < kUnits; ++q) {
        const int unit = unit0 + q, panel = unit >> 2, pair = (unit >> 1) & 1, g = (lane >> 3) + 4 * (unit & 1);
        v[q] = *reinterpret_cast<const uint4 *>(sC + (cs * 2 + panel) * C::kBlock + ((c * 2 + pair) * 32 + 4 * g + t) * 16);
      }
#pragma unroll
      for (int q = 0; q < kUnits; ++q) {
        // a panel that does not exist gives rows of the product that are not written
        const int unit = unit0 + q, panel = unit >> 2, pair = (unit >> 1) & 1, g = (lane >> 3) + 4 * (unit & 1);
        const uint32_t word[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
        uint32_t zeros = 0u;
        if constexpr (kZeros)
          zeros = *reinterpret_cast<const uint32_t *>(sC + (cs * 2 + panel) * C::kBlock + kW4CodeBytes + 128 * kGpb + (gi * 8 + g) * 8 + 4 * pair);
        uint8_t *dst = sA + stage * C::kABytes + (64 * panel + 32 * pair + g) * 128 + (((4 * cb + t) ^ g) << 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t p[4];
          w4_unpack<T>(word[i], kZeros ? w4_zero<T>(zeros, i) : w4_zero<T>(8), p);
          *reinterpret_cast<uint4 *>(dst + i * 1024) = make_uint4(p[0], p[1], p[2], p[3]);
        }
      }
      fence_proxy_async_shared();  // read by the tensor core
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&full[stage]);
        mbar_arrive(&empty_c[cs]);
      }
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------------- epilogue: this CTA's sums of a row and 64 (kTok) tokens
    pdl_wait();
    constexpr int kCols = kTok > 64 ? 64 : kTok;
    const int quarter = warp & 3, col0 = (warp - 4) / 4 * kCols, row = quarter * 32 + lane, r = row & 63;
    const uint32_t lanes = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + col0;
    const int at = (r & 7) * 8 + (r >> 4) * 2 + ((r >> 3) & 1);
    float sum[kCols];
#pragma unroll
    for (int j = 0; j < kCols; ++j) sum[j] = 0.f;
    int cs = 0;
    uint32_t cphase = 0, n = 0;
    for (int kb = kb0; ok && kb < kb1; ++kb) {
      ok = wait(&full_c[cs], cphase);  // the scales came by a copy
      const uint16_t *scales = reinterpret_cast<const uint16_t *>(sC + (cs * 2 + (row >> 6)) * C::kBlock + kW4CodeBytes);
#pragma unroll
      for (int gi = 0; gi < kGpb; ++gi) {
        if (!ok) break;
        const float s = row < 64 * mine ? T::up(scales[gi * 64 + at]) : 0.f;
        const uint32_t buf = n % C::kBufs;
        const int step = 2 * (kb - kb0) + (kGpb == 1 ? 0 : gi * 2 / kGpb);  // the group's (first) stage
        ok = wait(&done[step % C::kStages], step / C::kStages & 1);
        if (kGpb == 1) ok = ok && wait(&done[(step + 1) % C::kStages], (step + 1) / C::kStages & 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < kCols; c += 16) {
          uint32_t v[16];
          tmem_ld16(lanes + buf * kTok + c, v);
          tmem_ld_wait();
          if (c == kCols - 16) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[buf]);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) sum[c + i] = fmaf(__uint_as_float(v[i]), s, sum[c + i]);
        }
        ++n;
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty_c[cs]);
      if (++cs == C::kCodes) {
        cs = 0;
        cphase ^= 1;
      }
    }
    if (ok) {
      // every group has been read, so every MMA and copy of this CTA into the ring has completed
      float *part = reinterpret_cast<float *>(smem) + row;  // token j at part[128 j]
#pragma unroll
      for (int j = 0; j < kCols; ++j) part[128 * (col0 + j)] = sum[j];
    }
  }

  // ---------------------------------------------------------------- reduction over the ranks
  tc_fence_before();
  block_meet();
  if (splits > 1) cluster_meet();
  tc_fence_after();
  if (warp == 3) tmem_dealloc(tmem_base, C::kTmemCols);
  if (*abort_flag == 0) {
    const int live = min(kTok, args.M - m0);
    const uint32_t base = smem_u32(smem);
    for (int e = live * rank / splits * 128 + static_cast<int>(threadIdx.x); e < live * (rank + 1) / splits * 128; e += C::kThreads) {
      const int f = tile * 128 + (e & 127);
      const float s = cluster_sum(base + e * 4, splits);
      if (f < args.N) static_cast<uint16_t *>(args.y)[static_cast<int64_t>(m0 + (e >> 7)) * args.N + f] = T::one(s * power_of_two(W4Scale<T>::kRest));
    }
  }
  if (splits > 1) cluster_meet();  // no CTA leaves while another reads its sums
}

template <class T, int kGpb, bool kZeros, int kTok>
cudaError_t tc_as(const CUtensorMap &x, const W4Args &a, int splits, cudaStream_t s) {
  using C = TcCfg<kGpb, kZeros, kTok>;
  const cudaError_t e = allow_smem<w4_tc_kernel<T, kGpb, kZeros, kTok>>(static_cast<int>(C::kSmem));
  if (e != cudaSuccess) return e;
  return launch_clusters(w4_tc_kernel<T, kGpb, kZeros, kTok>, dim3(static_cast<unsigned>((a.N + 127) / 128 * splits), static_cast<unsigned>((a.M + kTok - 1) / kTok)),
                         C::kThreads, C::kSmem, splits, s, x, a, splits);
}

template <class T, int kGpb, bool kZeros>
cudaError_t tc_tok(const CUtensorMap &x, const W4Args &a, int tok, int splits, cudaStream_t s) {
  switch (tok) {
    case 32: return tc_as<T, kGpb, kZeros, 32>(x, a, splits, s);
    case 64: return tc_as<T, kGpb, kZeros, 64>(x, a, splits, s);
    case 128: return tc_as<T, kGpb, kZeros, 128>(x, a, splits, s);
  }
  return cudaErrorInvalidValue;
}
template <class T>
cudaError_t tc_group(const CUtensorMap &x, const W4Args &a, int group, bool zeros, int tok, int splits, cudaStream_t s) {
  if (group == 128) return zeros ? tc_tok<T, 1, true>(x, a, tok, splits, s) : tc_tok<T, 1, false>(x, a, tok, splits, s);
  if (group == 64) return zeros ? tc_tok<T, 2, true>(x, a, tok, splits, s) : tc_tok<T, 2, false>(x, a, tok, splits, s);
  return zeros ? tc_tok<T, 4, true>(x, a, tok, splits, s) : tc_tok<T, 4, false>(x, a, tok, splits, s);
}

}  // namespace

cudaError_t launch_w4_tc(const CUtensorMap &x, const W4Args &a, int dtype, int group, bool zeros, int tok, int splits,
                         cudaStream_t s) {
  return dtype == NVFP4_DT_BF16 ? tc_group<Bf16>(x, a, group, zeros, tok, splits, s) : tc_group<Fp16>(x, a, group, zeros, tok, splits, s);
}

}  // namespace nvfp4
