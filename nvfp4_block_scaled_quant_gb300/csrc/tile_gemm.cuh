// Tensor-bound GEMM on CTA pairs (tcgen05 cta_group::2) shared by the FP8 block-scaled linear
// and the gated linear's forward and backward products.
//
// One output tile per pair has 256 rows (128 per CTA, the lanes of its tensor memory) and 256 (or 128)
// accumulator columns.  A K block is 128 bytes of every operand row: each CTA stages 128 rows of A
// and half of the tile's rows of B per block (32 KB), a ring of kStages blocks deep.  A one-SM tile of 128 x 256
// would stage 48 KB for the same work: the L2 -> SM operand stream is what bounds tiles of this
// size, so the pair's sharing of B matters.
//
// Warps of each CTA: 0 = TMA producer, 1 (and 2 for FP8) = MMA issuer (the even CTA's, for both), 3 = tensor
// memory, 4..11 = epilogue (two per 32-lane quarter of tensor memory, half of the columns each).
//
//   Op::kFp8    A = xq (M, K) e4m3, B = wq (N, K) e4m3.  The scales change every 128 K, so every K
//               block is a product of its own: two issuers take the blocks in turn into an accumulator
//               each, and the epilogue warps add block * (sa[m, b] * sw[n / 128, b]) to fp32 registers
//               (128 columns per thread) while the next block runs.  Scaling in registers keeps the
//               scales arbitrary fp32 values; nothing is rounded until the output.
//               4096 x 7168 x 7168: 161 us, 2.6 PF/s.  A block takes 0.41 us where its MMAs take 0.26:
//               an accumulator's way to the epilogue and back (commit, wait, read, release, wait) is
//               longer than the other's MMAs.  Measured and left: four accumulators of 128 columns (two
//               issuers; 8 warps 200 us, 16 warps 175 us), 16 epilogue warps on 256 columns, two batches
//               of columns in flight, activation scales through a shared-memory ring.
//   Op::kGated  A = x (M, K), B = rows of Wg (even CTA) and the matching rows of Wu (odd CTA):
//               the first half of the accumulator's columns is g, the second u of the same outputs.
//   Op::kGrad   two products in one launch.  dx = dg Wg + du Wu: A = [dg | du] in two segments of K = I,
//               B = Wg, then Wu, read along their rows (MN-major B).  [dWg; dWu] = [dg | du]^T x: A and B
//               MN-major, K = tokens.  Their tiles differ in length, and either alone often leaves SMs idle in its
//               last wave, so a pair that has one tile of dx less than the others takes `early` tiles of
//               dW meanwhile.  With the activation's gradient, in one launch / two: 517 x 1536 x 2048 22.4 / 32.4 us,
//               2048 x 2048 x 4096 94 / 107, 700 x 7168 x 4096 118 / 141, 4096 x 7168 x 2048 274 / 275.
//
// Two of these launches never overlap.  On one stream they run in plain stream order, without programmatic
// dependent launch and without letting a successor start early (about 2 us per launch); on several
// streams each waits for the one launched before it (in_pair_turn).  An earlier form of the kernel whose launches
// overlapped, one taking over the SMs and tensor memory that the other leaves cluster by cluster, stopped making
// progress once in some thousand.  That form left commits and releases on their way to barriers of CTAs
// that had exited, freed a pair's tensor memory without waiting for the other CTA to have done so, and
// met at .aligned barriers with warps that might still be diverged; none of this is left, but which of it
// was the cause is not proven, so the overlap itself is kept out.
//
// Every mbarrier wait is bounded: a role that gives up raises NVFP4_DEVERR_PIPELINE_TIMEOUT, the copies in
// flight are given time to land, and every thread of the pair meets at the final cluster barrier.  The
// tensor-memory allocation, the cluster and block barriers and the register reallocation have no limit of their own:
// the allocation waits at most for CTAs of other kernels to leave the SM (its shared memory holds one of these), every
// thread reaches every barrier whatever its waits returned, and the register shares add up to the launch's.
#pragma once

#include <atomic>
#include <type_traits>

#include "mma16x8.cuh"

namespace nvfp4 {

enum class TileOp : int { kFp8 = 0, kGated = 1, kGrad = 2 };

struct TileArgs {
  int M, N;        // output rows and columns (kGated: N = I; kGrad: dx's, M = 0 without it)
  int k_blocks;    // 128-byte K blocks (kGrad: of one of dx's two segments)
  int dw_M, dw_k_blocks, early;  // kGrad: rows of [dWg; dWu] (0 without them), blocks of tokens, see above
  const float *sa; // kFp8: (K blocks, ld_sa) activation scales
  int64_t ld_sa;
  const float *sw; // kFp8: (ceil(N / 128), K blocks) weight scales
  void *out;       // 16-bit (M, N), row stride ldo
  void *dwg, *dwu; // kGrad: the weight gradients, (dw_M / 2, N) each, row stride ldo
  const float *unscale;  // kGrad, fp16: factor of the sums (the inverse of dg's and du's power of two)
  int64_t ldo;
  float *save;     // kGated: fp32 (M, 2N) pre-activations [g | u], or null
  uint32_t *err;
};

constexpr int kTRows = 256, kTHalf = 128;
// kCols accumulator columns of a tile, half of them staged by either CTA: 256, or 128 where 256 x 256
// tiles would leave SMs idle (tile_plan).
template <int kCols>
struct TileCfg {
  static constexpr int kStages = kCols == 256 ? 6 : 8;
  static constexpr int kABytes = kTHalf * 128;      // 128 rows x 128 bytes
  static constexpr int kBBytes = kCols / 2 * 128;   // kCols / 2 rows x 128 bytes
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr uint32_t kTmemCols = 2 * kCols;  // two accumulators
  static constexpr int kStoreBytes = 8 * 32 * 36;   // kFp8: a warp's 32 rows of 16 columns on their way out
  static constexpr size_t kSmem = 1024 + kRing + 256 + kStoreBytes;
  static_assert(kSmem <= 232448, "per-block shared memory limit");
  static_assert((2 * kStages + 4) * 8 + 8 <= 256, "barrier region");
};
constexpr int kTAllocWarp = 3;  // owns the tensor memory; it has no other role, so it is never diverged
constexpr int kTEpiWarp0 = 4;  // epilogue warps start on a multiple of four: a warp reads lane quarter warp % 4
template <TileOp kOp>
constexpr int kTEpiWarps = 8;
template <TileOp kOp>
constexpr int kTThreads = (kTEpiWarp0 + kTEpiWarps<kOp>)*32;
template <TileOp kOp>
constexpr int kTIssuers = kOp == TileOp::kFp8 ? 2 : 1;
// kFp8: registers per thread.  The launch gives every warp 168 (three warps on each quarter of an
// SM); the epilogue's 128 sums, scales and accumulator columns in flight take more, which the first four
// warps give up.
constexpr int kTLaunchRegs = 168, kTLightRegs = 56, kTEpiRegs = 224;
static_assert(kTEpiWarp0 * kTLightRegs + kTEpiWarps<TileOp::kFp8> * kTEpiRegs <=
                  (kTEpiWarp0 + kTEpiWarps<TileOp::kFp8>)*kTLaunchRegs,
              "register split within what the block was launched with");
constexpr int kAhead = 4;             // kFp8: K blocks that a thread's scales are fetched ahead
constexpr int kTGroupM = 8;           // m tiles walked together, so that a wave shares rows of B in L2
template <TileOp kOp, class T, int kAct, int kTCols>
__global__ void __launch_bounds__(kTThreads<kOp>, 1)
    tile_gemm_kernel(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmA1,
                     const __grid_constant__ CUtensorMap tmB0, const __grid_constant__ CUtensorMap tmB1,
                     const __grid_constant__ CUtensorMap tmA2, const __grid_constant__ CUtensorMap tmB2,
                     const TileArgs args) {
  using C = TileCfg<kTCols>;
  constexpr int kBRows = kTCols / 2;  // rows of B staged by a CTA
  constexpr bool kFp8 = kOp == TileOp::kFp8;
  constexpr bool kGrad = kOp == TileOp::kGrad;
  constexpr int kOutCols = kOp == TileOp::kGated ? kBRows : kTCols;  // output columns of a tile
  constexpr uint32_t kFmt = kFp8 ? 0u : (T::kCode == NVFP4_DT_BF16 ? 1u : 0u);

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint8_t *sA = smem;
  uint8_t *sB = sA + C::kStages * C::kABytes;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kRing);  // used in the even CTA
  uint64_t *empty = full + C::kStages;
  uint64_t *tfull = empty + C::kStages;   // [2]
  uint64_t *tempty = tfull + 2;     // [2], used in the even CTA
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(tempty + 2);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
  uint16_t *s_store = reinterpret_cast<uint16_t *>(smem + C::kRing + 256);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * 8);  // the eight warps of each CTA that read it
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tmA0);
    prefetch_tensormap(&tmB0);
  }
  __syncwarp();
  if (warp == kTAllocWarp) {
    tmem_alloc_pair(tmem_holder, C::kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  block_meet();
  cluster_meet();  // both CTAs' barriers are initialised and their tensor memory allocated
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  const int m_tiles = (args.M + kTRows - 1) / kTRows, dw_m_tiles = kGrad ? (args.dw_M + kTRows - 1) / kTRows : 0;
  const int n_tiles = (args.N + kOutCols - 1) / kOutCols;
  const int total = m_tiles * n_tiles, dw_total = dw_m_tiles * n_tiles;
  const int k_blocks = args.k_blocks * (kGrad ? 2 : 1);
  const int clusters = static_cast<int>(gridDim.x) / 2, cluster_id = static_cast<int>(blockIdx.x) / 2;
  // after a wait that gave up: the time that copies and MMAs in flight need, many times over
  auto settle = [] {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 10000000ull) {
    }
  };
  struct Tile {
    int mt, nt;
    bool dw;  // kGrad: a tile of [dWg; dWu]
  };
  auto place = [&](int idx, int m_tiles, Tile &t) {
    const int per_group = kTGroupM * n_tiles, g = idx / per_group, in = idx - g * per_group;
    const int rows = min(kTGroupM, m_tiles - g * kTGroupM);
    t.nt = in / rows;
    t.mt = g * kTGroupM + (in - t.nt * rows);
  };
  // The tile at a pair's step of its walk, from `first` in steps of `step`; false past its last.  The pairs take the
  // tiles in turn.  kGrad: dx's first; the pairs behind the last one of dx's final round then take `early`
  // rounds of dW's, and the turns go on from them.
  const int first = kGrad ? 0 : cluster_id, step = kGrad ? 1 : clusters;
  auto tile_of = [&](int at, Tile &t) {
    t.dw = false;
    if constexpr (!kGrad) {
      if (at >= total) return false;
      place(at, m_tiles, t);
      return true;
    } else {
      int j = at, idx = cluster_id + j * clusters;
      if (idx < total) {
        place(idx, m_tiles, t);
        return true;
      }
      t.dw = true;
      const int behind = total % clusters, rest = clusters - behind;
      j -= total / clusters + (cluster_id < behind ? 1 : 0);
      if (cluster_id >= behind && j < args.early) {
        idx = cluster_id - behind + j * rest;
      } else {
        if (cluster_id >= behind) j -= args.early;
        const int turn = cluster_id >= behind ? cluster_id - behind : cluster_id + rest;
        idx = min(dw_total, args.early * rest) + turn + j * clusters;
      }
      if (idx >= dw_total) return false;
      place(idx, dw_m_tiles, t);
      return true;
    }
  };

  if constexpr (kFp8) {
    if (warp < kTEpiWarp0)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTLightRegs));
    else
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTEpiRegs));
  }
  if (warp == 0) {
    // -------------------------------------------------------------- TMA producer (one elected lane copies)
    const uint64_t pol = policy_evict_normal();
    const uint32_t full_leader = cluster_addr(full, 0);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    // K block `kb` of both operands.  The form of A is a constant of each loop: a branch and a choice of the map at
    // every block made the producer the kernel's limit (dx of 517 x 1536 x 2048 25.7 us instead of 21.3).
    auto load = [&](const CUtensorMap *mapA, const CUtensorMap *mapB, int kb, int a_row, int b_row, auto dw) {
      constexpr bool kAMn = decltype(dw)::value;
      ok = mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, args.err, kPipelineTimeoutNs);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      if (elect_one()) {
        // both CTAs' copies complete on the even CTA's barrier, which expects all of them
        if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * C::kStageBytes);
        const uint32_t bar = full_leader + stage * 8;
        uint8_t *a = sA + stage * C::kABytes, *b = sB + stage * C::kBBytes;
        if constexpr (kAMn) {  // 64 K rows of 64 elements, two boxes side by side along M
          tma_load_2d_pair(a, mapA, a_row * 2, kb * 64, bar, pol);
          tma_load_2d_pair(a + 8192, mapA, a_row * 2 + 128, kb * 64, bar, pol);
        } else {
          tma_load_2d_pair(a, mapA, kb * 128, a_row, bar, pol);
        }
        if constexpr (kGrad) {
          tma_load_2d_pair(b, mapB, b_row * 2, kb * 64, bar, pol);
          if constexpr (kBRows == 128) tma_load_2d_pair(b + 8192, mapB, b_row * 2 + 128, kb * 64, bar, pol);
        } else {
          tma_load_2d_pair(b, mapB, kb * 128, b_row, bar, pol);
        }
      }
      __syncwarp();
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1;
      }
    };
    Tile t;
    for (int at = first; ok && tile_of(at, t); at += step) {
      const int a_row = t.mt * kTRows + static_cast<int>(rank) * kTHalf;
      const int b_row = kOp == TileOp::kGated ? t.nt * kBRows : t.nt * kTCols + static_cast<int>(rank) * kBRows;
      if constexpr (kGrad) {
        if (t.dw) {
          for (int kb = 0; ok && kb < args.dw_k_blocks; ++kb) load(&tmA2, &tmB2, kb, a_row, b_row, std::true_type());
        } else {
          for (int kb = 0; ok && kb < args.k_blocks; ++kb) load(&tmA0, &tmB0, kb, a_row, b_row, std::false_type());
          for (int kb = 0; ok && kb < args.k_blocks; ++kb) load(&tmA1, &tmB1, kb, a_row, b_row, std::false_type());
        }
      } else {
        const CUtensorMap *mapB = kOp == TileOp::kGated && rank ? &tmB1 : &tmB0;
        for (int kb = 0; ok && kb < k_blocks; ++kb) load(&tmA0, mapB, kb, a_row, b_row, std::false_type());
      }
    }
    // Neither CTA may exit with a commit on its way to one of its barriers (the commits of the even
    // CTA's issuer arrive on both CTAs'): the ring is followed until every stage is free again.
    for (int i = 0; ok && i < C::kStages; ++i) {
      ok = mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, args.err, kPipelineTimeoutNs);
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (!ok) settle();  // copies in flight may complete on the other CTA's barrier
  } else if (warp < kTEpiWarp0) {
    if (rank == 0 && warp <= kTIssuers<kOp>) {
      // ------------------------------------------------------------ MMA issuers
      // The whole warp waits and one elected lane issues: in an elect.sync branch an MMA takes its
      // issuer about 32 cycles, from a `lane == 0` branch about its execution time, and the waits
      // and commits between K blocks then leave the tensor pipe idle.
      const uint32_t a0 = smem_u32(sA), b0 = smem_u32(sB);
      // K-major rows of 128 bytes: 8-row groups 1024 bytes apart, a K step is 32 bytes on.
      // MN-major boxes (64 elements x 64 K rows): boxes 8192 bytes apart along MN, 8-K groups 1024
      // bytes apart, a K step of 16 rows is 2048 bytes on.
      constexpr int kIssuers = kTIssuers<kOp>;
      const int iss = warp - 1;
      int stage = iss;
      uint32_t phase = 0;
      uint32_t acc = iss;  // the accumulator's turn: the block (kFp8) or the tile
      bool ok = true;
      // block `it` of a tile, its last if `done`
      auto issue = [&](int it, bool done, auto dw) {
        constexpr bool kAMn = decltype(dw)::value;
        constexpr uint32_t kAStep = kAMn ? 2048 / 16 : 32 / 16, kBStep = kGrad ? 2048 / 16 : 32 / 16;
        constexpr uint32_t kIdesc = mma_idesc(kFmt, kAMn, kGrad, kTRows, kTCols);
        if (kFp8 || it == 0)
          ok = mbar_wait_bounded_cluster(&tempty[acc & 1], ((acc >> 1) & 1) ^ 1, abort_flag, args.err, kPipelineTimeoutNs);
        ok = ok && mbar_wait_bounded_cluster(&full[stage], phase, abort_flag, args.err, kPipelineTimeoutNs);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t ad = smem_desc(a0 + stage * C::kABytes, kAMn ? 8192 : 16, 1024, 2);
          const uint64_t bd = smem_desc(b0 + stage * C::kBBytes, kGrad ? 8192 : 16, 1024, 2);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            tc_mma<kFp8, true>(tmem_base + (acc & 1) * kTCols, ad + j * kAStep, bd + j * kBStep, kIdesc,
                               kFp8 ? j != 0 : (it | j) != 0);
          tc_commit_pair(&empty[stage], 0x3);
          if (done) tc_commit_pair(&tfull[acc & 1], 0x3);
        }
        __syncwarp();
        if (done) acc += kIssuers;
        if ((stage += kIssuers) >= C::kStages) {
          stage -= C::kStages;
          phase ^= 1;
        }
      };
      if constexpr (kFp8) {
        // the two issuers take the launch's blocks in turn, issuer i into accumulator i
        const int tiles = cluster_id < total ? (total - 1 - cluster_id) / clusters + 1 : 0;
        const int64_t blocks = static_cast<int64_t>(tiles) * k_blocks;
        for (int64_t g = iss; ok && g < blocks; g += kIssuers) issue(0, true, std::false_type());
      } else {
        Tile t;
        for (int at = first; ok && tile_of(at, t); at += step) {
          if constexpr (kGrad) {
            if (t.dw) {
              for (int it = 0; ok && it < args.dw_k_blocks; ++it) issue(it, it == args.dw_k_blocks - 1, std::true_type());
              continue;
            }
          }
          for (int it = 0; ok && it < k_blocks; ++it) issue(it, it == k_blocks - 1, std::false_type());
        }
      }
      // Every accumulator has come back, so every MMA has completed before the pair frees its tensor
      // memory, and no release of the other CTA's epilogue is on its way to this CTA's barriers.
      for (int64_t turn = static_cast<int64_t>(acc) - 2; ok && turn < acc; ++turn)
        if (turn >= 0 && (!kFp8 || (turn & 1) == iss))
          ok = mbar_wait_bounded_cluster(&tempty[turn & 1], static_cast<uint32_t>(turn >> 1) & 1, abort_flag, args.err,
                                         kPipelineTimeoutNs);
      if (!ok) settle();
    }
  } else {
    // -------------------------------------------------------------- epilogue
    const int quarter = warp & 3, half = (warp - kTEpiWarp0) >> 2;
    const uint32_t tempty_leader = cluster_addr(tempty, 0);
    const uint32_t lanes = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    uint32_t acc = 0;
    bool ok = true;
    auto wait_acc = [&]() {
      ok = mbar_wait_bounded(&tfull[acc & 1], (acc >> 1) & 1, abort_flag, args.err, kPipelineTimeoutNs);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      return ok;
    };
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(tempty_leader + (acc & 1) * 8);
      ++acc;
    };
    const bool vec = (args.ldo & 7) == 0;
    constexpr bool kUnscale = kGrad && T::kCode == NVFP4_DT_FP16;
    const float unscale = kUnscale ? __ldg(args.unscale) : 1.f;
    // kFp8: the sums of this thread's row, kBRows columns from out_n0 on
    float sum[kFp8 ? kBRows : 1];
    int out_row = 0, out_n0 = 0;
    auto store_tile = [&]() {
      if constexpr (kFp8) {
#pragma unroll
        for (int c = 0; c < kBRows / 16; ++c) {
          float v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = sum[c * 16 + i];
          const int left = args.N - out_n0 - c * 16;
          if (vec) {
            if (out_row < args.M)
              store16<T>(static_cast<uint16_t *>(args.out) + out_row * args.ldo + out_n0 + c * 16, v, left, true);
          } else if (left > 0) {
            // rows of any alignment: through shared memory, so that 16 lanes write 16 consecutive
            // elements (a lane per row would touch 32 sectors with every 2-byte store)
            uint16_t *mine = s_store + (warp - kTEpiWarp0) * 32 * 18;
            uint32_t *w = reinterpret_cast<uint32_t *>(mine + lane * 18);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = T::pack(v[2 * i], v[2 * i + 1]);
            __syncwarp();
            const int at = lane & 15;
            for (int r = lane >> 4; r < 32; r += 2) {
              const int row = out_row - lane + r;
              if (row < args.M && at < left)
                static_cast<uint16_t *>(args.out)[row * args.ldo + out_n0 + c * 16 + at] = mine[r * 18 + at];
            }
            __syncwarp();
          }
        }
      }
    };
    Tile tile;
    for (int at = first; ok && tile_of(at, tile); at += step) {
      const int nt = tile.nt;
      const int row = tile.mt * kTRows + static_cast<int>(rank) * kTHalf + quarter * 32 + lane;
      const bool row_ok = row < (kGrad && tile.dw ? args.dw_M : args.M);
      if constexpr (kFp8) {
        const int n0 = nt * kTCols + half * kBRows;  // a warp's columns share one weight scale
        // Scales are fetched ahead: under the operand stream a load takes longer than a block.  The
        // thread's row's activation scales kAhead blocks ahead (the loop is unrolled, so that no
        // register in flight is moved); a lane holds every 32nd weight scale.  Rows past M and
        // columns past N read the last one's.
        const float *sa = args.sa + min(row, args.M - 1);
        const float *sw = args.sw + static_cast<int64_t>(min(n0, args.N - 1) / 128) * k_blocks;
        float w = ld_early(sw + min(lane, k_blocks - 1)), a[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) a[u] = ld_early(sa + min(u, k_blocks - 1) * args.ld_sa);
        if (at != first) store_tile();  // the previous tile, while this one's first block is made
        out_row = row;
        out_n0 = n0;
#pragma unroll
        for (int i = 0; i < kBRows; ++i) sum[i] = 0.f;
        for (int kb0 = 0; ok && kb0 < k_blocks; kb0 += kAhead) {
          if ((kb0 & 31) == 0 && kb0) w = ld_early(sw + min(kb0 + lane, k_blocks - 1));
#pragma unroll
          for (int u = 0; u < kAhead; ++u) {
            if (kb0 + u >= k_blocks) break;
            const float f = a[u] * __shfl_sync(0xffffffffu, w, (kb0 + u) & 31);
            a[u] = ld_early(sa + min(kb0 + u + kAhead, k_blocks - 1) * args.ld_sa);
            if (!wait_acc()) break;
            const uint32_t t = lanes + (acc & 1) * kTCols + half * kBRows;
            // scalar FMAs: the packed form (fma.rn.f32x2) has no higher rate here and cost 16% more time
#pragma unroll
            for (int c = 0; c < kBRows / 16; ++c) {
              uint32_t r[16];
              tmem_ld16(t + c * 16, r);
              tmem_ld_wait();
              if (c == kBRows / 16 - 1) release();
#pragma unroll
              for (int i = 0; i < 16; ++i) sum[c * 16 + i] = fmaf(__uint_as_float(r[i]), f, sum[c * 16 + i]);
            }
          }
        }
        if (!ok) break;
      } else if constexpr (kOp == TileOp::kGated) {
        if (!wait_acc()) break;
        const int n0 = nt * kBRows + half * (kBRows / 2);
        const uint32_t t = lanes + (acc & 1) * kTCols + half * (kBRows / 2);
        uint16_t *dst = static_cast<uint16_t *>(args.out) + row * args.ldo + n0;
        float *save = args.save ? args.save + static_cast<int64_t>(row) * 2 * args.N + n0 : nullptr;
#pragma unroll
        for (int c = 0; c < kBRows / 32; ++c) {
          uint32_t g[16], u[16];
          tmem_ld16(t + c * 16, g);
          tmem_ld16(t + kBRows + c * 16, u);
          tmem_ld_wait();
          if (c == kBRows / 32 - 1) release();
          const int left = args.N - n0 - c * 16;
          if (row_ok && left > 0) {
            float h[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) h[i] = act_fwd<kAct>(__uint_as_float(g[i])) * __uint_as_float(u[i]);
            store16<T>(dst + c * 16, h, left, vec);
            if (save) {  // N % 8 == 0: whole groups of 8 columns, a sector each, exist or do not
#pragma unroll
              for (int i = 0; i < 16; i += 8)
                if (i < left) {
                  st_global_v8(save + c * 16 + i, reinterpret_cast<const uint32_t (&)[8]>(g[i]));
                  st_global_v8(save + args.N + c * 16 + i, reinterpret_cast<const uint32_t (&)[8]>(u[i]));
                }
            }
          }
          __syncwarp();
        }
      } else {
        if (!wait_acc()) break;
        const int n0 = nt * kTCols + half * kBRows;
        const uint32_t t = lanes + (acc & 1) * kTCols + half * kBRows;
        const int split = args.dw_M / 2;  // rows of dWg
        void *out = !tile.dw ? args.out : row < split ? args.dwg : args.dwu;
        uint16_t *dst = static_cast<uint16_t *>(out) + (tile.dw && row >= split ? row - split : row) * args.ldo + n0;
#pragma unroll
        for (int c = 0; c < kBRows / 16; ++c) {
          uint32_t r[16];
          __syncwarp();
          tmem_ld16(t + c * 16, r);
          tmem_ld_wait();
          if (c == kBRows / 16 - 1) release();
          float v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = kUnscale ? __uint_as_float(r[i]) * unscale : __uint_as_float(r[i]);
          if (row_ok) store16<T>(dst + c * 16, v, args.N - n0 - c * 16, vec);
        }
      }
    }
    if (ok && cluster_id < total) store_tile();
  }

  tc_fence_before();
  block_meet();
  cluster_meet();  // the pair's MMAs have drained and both epilogues have read their accumulators
  tc_fence_after();
  if (warp == kTAllocWarp) tmem_dealloc_pair(tmem_base, C::kTmemCols);
  // Freeing a pair's tensor memory takes both CTAs: neither leaves before the other has done it.
  cluster_meet();
}

// Clusters of two that fit on the current device at once (0 if the query fails), and the launch.
template <class K>
int tile_gemm_max_clusters(K kernel, int threads, size_t smem) {
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
    return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * 1024);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) return 0;
  return n;
}

template <TileOp kOp, class T, int kAct, int kTCols>
cudaError_t launch_tile_gemm_cols(const CUtensorMap &a0, const CUtensorMap &a1, const CUtensorMap &b0,
                                  const CUtensorMap &b1, const CUtensorMap &a2, const CUtensorMap &b2,
                                  const TileArgs &args, cudaStream_t s) {
  using C = TileCfg<kTCols>;
  auto kernel = tile_gemm_kernel<kOp, T, kAct, kTCols>;
  static std::atomic<int> fit[64];  // per device; the kernel's shared-memory limit is set with the query
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int n = fit[dev].load();
  if (n <= 0) {
    n = tile_gemm_max_clusters(kernel, kTThreads<kOp>, C::kSmem);
    if (n <= 0) {
      const cudaError_t last = cudaGetLastError();
      return last != cudaSuccess ? last : cudaErrorLaunchOutOfResources;
    }
    fit[dev].store(n);
  }
  const int out_cols = kOp == TileOp::kGated ? kTCols / 2 : kTCols;
  const int64_t n_tiles = (static_cast<int64_t>(args.N) + out_cols - 1) / out_cols;
  const int64_t tiles = ((static_cast<int64_t>(args.M) + kTRows - 1) / kTRows +
                         (kOp == TileOp::kGrad ? (static_cast<int64_t>(args.dw_M) + kTRows - 1) / kTRows : 0)) * n_tiles;
  // a balanced grid: every wave of equal tiles, the last included, is (nearly) full
  const int64_t waves = (tiles + n - 1) / n;
  const int clusters = static_cast<int>(kOp == TileOp::kGrad ? (tiles < n ? tiles : n) : (tiles + waves - 1) / waves);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * clusters);
  cfg.blockDim = dim3(kTThreads<kOp>);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a0, a1, b0, b1, a2, b2, args);
}

// cols: 256 or 128 accumulator columns per tile; B's tensor maps have boxes of cols / 2 rows
// (K-major) or 64 columns (MN-major).
template <TileOp kOp, class T, int kAct>
cudaError_t launch_tile_gemm_as(const CUtensorMap &a0, const CUtensorMap &a1, const CUtensorMap &b0,
                                const CUtensorMap &b1, const CUtensorMap &a2, const CUtensorMap &b2,
                                const TileArgs &args, int cols, cudaStream_t s) {
  return cols == 256 ? launch_tile_gemm_cols<kOp, T, kAct, 256>(a0, a1, b0, b1, a2, b2, args, s)
                     : launch_tile_gemm_cols<kOp, T, kAct, 128>(a0, a1, b0, b1, a2, b2, args, s);
}

}  // namespace nvfp4
