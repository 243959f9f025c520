// Weight-streaming GEMM for few rows of activations (decode and small batches), shared by the FP8
// block-scaled linear and the gated linear's forward.
//
// With few tokens the product is bound by the bytes of the weights, so the operands are swapped:
// 128 weight rows (output features) are the MMA's M = 128 and kTok tokens its N, and the reduction
// is split over the CTAs of a cluster so that enough weight bytes are in flight on every SM even
// where there are few 128-row tiles.  A stage of the ring is one 128-byte K block: 128 weight rows
// (kGated: 128 rows of Wg and 128 of Wu), kTok token rows, and for FP8 the block's token scales.
// Two CTAs fit on an SM.  (Measured and left: a ring twice as deep and one CTA per SM for launches of at
// most one CTA per SM.  A cluster of eight then needs eight whole SMs of one GPC: one token 7168 -> 2 x
// 2048 in bf16 took 22 us instead of 16.)
//
// The CTAs of a cluster hold partial sums of the same outputs; each leaves its partial in its own
// shared memory, and after a cluster barrier each adds its share of the token columns over all
// ranks in rank order (a fixed order: repeated calls give identical bits) and writes the outputs.
//
// FP8: the product of one K block goes to one of kBufs accumulators, and the epilogue warps add it
// to fp32 registers times sw[tile, b] * sa[b, token] (a 128-row weight tile has one scale per block).
//
// kQuant (FP8, tiles of at most 32 tokens): four more warps quantise the 16-bit activations into the ring
// themselves, with the quantiser kernel's arithmetic, so that a decoded token takes one launch.  Every
// CTA quantises its K blocks of all tokens; that pays while the tokens are few.
//
// Warps: 0 = TMA producer, 1 = MMA issuer, 2..5 = epilogue (one 32-lane quarter of tensor memory
// each), 6..9 = quantisers (kQuant).  Every wait is bounded, as in the tile GEMM.
#pragma once

#include <atomic>

#include "fp8_encode.cuh"
#include "mma16x8.cuh"

namespace nvfp4 {

struct StreamArgs {
  int M, N;        // tokens, output features (kGated: N = I)
  int k_blocks;    // 128-byte K blocks
  const float *sa; // FP8: (K blocks, ld_sa) activation scales
  int64_t ld_sa;   // a multiple of 4
  const float *sw; // FP8: (ceil(N / 128), K blocks)
  void *out;       // 16-bit (M, N), row stride ldo
  int64_t ldo;
  float *save;     // kGated: fp32 (M, 2N) [g | u], or null
  const void *x;   // kQuant: 16-bit activations (M, K), row stride ldx
  int64_t ldx;
  int K;           // kQuant
  uint32_t *err;
};

template <bool kFp8, int kTok, bool kQuant>
struct StreamCfg {
  static constexpr int kOperands = kFp8 ? 1 : 2;  // weight tiles per stage (gate and up)
  static constexpr int kWBytes = 128 * 128;
  static constexpr int kXBytes = kTok * 128;
  static constexpr int kSBytes = kFp8 ? kTok * 4 : 0;
  static constexpr int kStageBytes = kOperands * kWBytes + kXBytes;
  static constexpr int kStages = 104 * 1024 / (kStageBytes + kSBytes);
  static constexpr int kQuantWarps = kQuant ? 4 : 0;
  static constexpr int kThreads = 192 + kQuantWarps * 32;
  static constexpr int kBufs = kFp8 ? (kTok <= 64 ? 4 : 2) : 1;
  static constexpr int kCols = kFp8 ? kBufs * kTok : 2 * kTok;  // accumulator columns
  static constexpr uint32_t kTmemCols = kCols <= 32 ? 32 : kCols <= 64 ? 64 : kCols <= 128 ? 128 : 256;
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kPartialBytes = kOperands * kTok * 128 * 4;  // over the ring, once it is drained
  static constexpr size_t kSmem = kRing + kStages * kSBytes + 256;
  static_assert(kPartialBytes <= kRing, "the partial sums fit where the ring was");
  static_assert(kCols <= 256, "two CTAs share the SM's 512 tensor-memory columns");
  static_assert(2 * (kSmem + 1024) <= 233472, "two CTAs per SM");
  static_assert(!kQuant || (kFp8 && kTok <= 32), "a quantiser holds all tokens of a K block in registers");
  static_assert((2 * kStages + 2 * kBufs) * 8 + 8 <= 256, "barrier region");
  static_assert(kTok % 16 == 0 && kStages >= 2, "MMA N and ring");
};

constexpr int kStreamMaxSplit = 8;  // portable cluster size

// Quantising warps that share a K block of `rows` tokens, eight each (the last tile's rows may be fewer)
__device__ __forceinline__ int quant_share(int rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }

template <bool kFp8, class T, int kAct, int kTok, bool kQuant>
__global__ void __launch_bounds__(StreamCfg<kFp8, kTok, kQuant>::kThreads, 2)
    stream_gemm_kernel(const __grid_constant__ CUtensorMap tmW0, const __grid_constant__ CUtensorMap tmW1,
                       const __grid_constant__ CUtensorMap tmX, const StreamArgs args, const int splits) {
  using C = StreamCfg<kFp8, kTok, kQuant>;
  constexpr uint32_t kFmt = kFp8 ? 0u : (T::kCode == NVFP4_DT_BF16 ? 1u : 0u);
  constexpr uint32_t kIdesc = mma_idesc(kFmt, false, false, 128, kTok);

  extern __shared__ __align__(1024) uint8_t smem[];  // used as declared: its accesses are known to be shared ones
  uint8_t *sW = smem;                                            // stages x operands x 16 KiB
  uint8_t *sX = sW + C::kStages * C::kOperands * C::kWBytes;     // stages x token rows
  float *sS = reinterpret_cast<float *>(sX + C::kStages * C::kXBytes);  // stages x token scales
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kRing + C::kStages * C::kSBytes);
  uint64_t *empty = full + C::kStages;
  uint64_t *tfull = empty + C::kStages;   // [kBufs]
  uint64_t *tempty = tfull + C::kBufs;    // [kBufs]
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(tempty + C::kBufs);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(blockIdx.x) % splits, tile = static_cast<int>(blockIdx.x) / splits;
  const int m0 = static_cast<int>(blockIdx.y) * kTok;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], kQuant ? 1 + quant_share(min(kTok, args.M - m0)) : 1);
      // FP8: the epilogue also reads the stage's token scales
      mbar_init(&empty[s], kFp8 ? 5 : 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 4);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tmW0);
    if constexpr (!kQuant) prefetch_tensormap(&tmX);
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc(tmem_holder, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  block_meet();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  pdl_wait();
  pdl_trigger();

  // this rank's K blocks
  const int kb0 = static_cast<int>(static_cast<int64_t>(args.k_blocks) * rank / splits);
  const int kb1 = static_cast<int>(static_cast<int64_t>(args.k_blocks) * (rank + 1) / splits);
  auto settle = [] {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 10000000ull) {
    }
  };
  constexpr int kMaxCols = kTok;
  float acc[kFp8 ? kMaxCols : 1];

  if (warp == 0) {
    // -------------------------------------------------------------- TMA producer (one elected lane copies)
    const uint64_t pol_w = policy_evict_first(), pol_x = policy_evict_last();
    // token scales that exist from m0 on, rounded up to whole 16 bytes (a row of scales is padded)
    const uint32_t s_bytes = kFp8 && !kQuant ? static_cast<uint32_t>(min(kTok, (args.M - m0 + 3) & ~3)) * 4u : 0u;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      ok = mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, args.err, kPipelineTimeoutNs);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(&full[stage], C::kStageBytes - (kQuant ? C::kXBytes : 0) + s_bytes);
        uint8_t *w = sW + stage * C::kOperands * C::kWBytes;
        tma_load_2d(w, &tmW0, kb * 128, tile * 128, &full[stage], pol_w);
        if constexpr (!kFp8) tma_load_2d(w + C::kWBytes, &tmW1, kb * 128, tile * 128, &full[stage], pol_w);
        if constexpr (!kQuant) tma_load_2d(sX + stage * C::kXBytes, &tmX, kb * 128, m0, &full[stage], pol_x);
        if constexpr (kFp8 && !kQuant) bulk_load(sS + stage * kTok, args.sa + kb * args.ld_sa + m0, s_bytes, &full[stage], pol_x);
      }
      __syncwarp();
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    // no commit is on its way to a barrier of this CTA when it exits
    for (int i = 0; ok && i < C::kStages; ++i) {
      ok = mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, args.err, kPipelineTimeoutNs);
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (!ok) settle();
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA issuer (one elected lane issues)
    const uint32_t w0 = smem_u32(sW), x0 = smem_u32(sX);
    int stage = 0;
    uint32_t phase = 0, n = 0;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      const uint32_t buf = kFp8 ? n % C::kBufs : 0;
      if (kFp8) ok = mbar_wait_bounded(&tempty[buf], ((n / C::kBufs) & 1) ^ 1, abort_flag, args.err, kPipelineTimeoutNs);
      ok = ok && mbar_wait_bounded(&full[stage], phase, abort_flag, args.err, kPipelineTimeoutNs);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t xd = smem_desc(x0 + stage * C::kXBytes, 16, 1024, 2);
#pragma unroll
        for (int o = 0; o < C::kOperands; ++o) {
          const uint64_t wd = smem_desc(w0 + (stage * C::kOperands + o) * C::kWBytes, 16, 1024, 2);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            tc_mma<kFp8, false>(tmem_base + (kFp8 ? buf : o) * kTok, wd + 2 * j, xd + 2 * j, kIdesc,
                                kFp8 ? j != 0 : (kb != kb0 || j != 0));
        }
        tc_commit(&empty[stage]);
        if (kFp8 || kb == kb1 - 1) tc_commit(&tfull[buf]);
      }
      __syncwarp();
      ++n;
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (!ok) settle();
  } else if (kQuant && warp >= 6) {
    // -------------------------------------------------------------- quantisers
    // A warp takes eight tokens of a K block, two at a time (16 lanes hold one token's 128 elements),
    // so the four warps work on four, two or one blocks at once, for up to 8, 16 or more tokens: the
    // latency of a block, a few hundred cycles of dependent steps, is shared by the blocks in work (one
    // token 7168 -> 7168: 9.1 us, with the four warps on one block 15.5).  A register is loaded again,
    // for the warp's next block, as soon as it is encoded.  Columns of tokens past M are left as they
    // are: they feed no output.
    if constexpr (kQuant) {
      constexpr int kHold = 4;
      static_assert(C::kStages >= C::kQuantWarps, "a warp's stages wrap at most once per step");
      const int share = quant_share(min(kTok, args.M - m0)), step = C::kQuantWarps / share;
      const int gl = lane & 15, row0 = (warp - 6) % share * 8 + (lane >> 4);
      const uint16_t *x = static_cast<const uint16_t *>(args.x) + (m0 + row0) * args.ldx + gl * 8;
      auto load = [&](int kb, int q) {
        return m0 + row0 + q * 2 < args.M && kb < kb1 && kb * 128 + gl * 8 < args.K
                   ? __ldg(reinterpret_cast<const uint4 *>(x + q * 2 * args.ldx + kb * 128))
                   : make_uint4(0u, 0u, 0u, 0u);
      };
      int stage = (warp - 6) / share;
      uint32_t phase = 0;
      uint4 v[kHold];
#pragma unroll
      for (int q = 0; q < kHold; ++q) v[q] = load(kb0 + stage, q);
      for (int kb = kb0 + stage; kb < kb1; kb += step) {
        bool ok = mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, args.err, kPipelineTimeoutNs);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
#pragma unroll
        for (int q = 0; q < kHold; ++q) {
          const int row = row0 + q * 2;
          const bool mine = m0 + row < args.M;
          if (__any_sync(0xffffffffu, mine)) {
            uint32_t a = max_abs16(v[q]);
#pragma unroll
            for (int o = 8; o; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
            const float sc = scale_of<T>(a);
            if (mine) {  // rows of 128 bytes, 16-byte chunks swizzled by the row
              uint8_t *d = sX + stage * C::kXBytes + row * 128 + (((gl >> 1) ^ (row & 7)) << 4) + (gl & 1) * 8;
              *reinterpret_cast<uint2 *>(d) = encode8<T>(v[q], sc);
              if (gl == 0) sS[stage * kTok + row] = sc;
            }
          }
          v[q] = load(kb + step, q);
        }
        fence_proxy_async_shared();  // the codes are read by the tensor core
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[stage]);
        stage += step;
        if (stage >= C::kStages) {
          stage -= C::kStages;
          phase ^= 1;
        }
      }
    }
  } else {
    // -------------------------------------------------------------- epilogue: this CTA's sums
    const int quarter = warp & 3;
    const uint32_t lanes = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    float *part = reinterpret_cast<float *>(smem) + quarter * 32 + lane;  // column j at part[128 j]
    bool ok = true;
    if constexpr (kFp8) {
#pragma unroll
      for (int j = 0; j < kTok; ++j) acc[j] = 0.f;
      const float *sw = args.sw + static_cast<int64_t>(tile) * args.k_blocks;
      float next_w = __ldg(sw + kb0);
      int stage = 0;
      uint32_t phase = 0, n = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++n) {
        const float w = next_w;
        if (kb + 1 < kb1) next_w = __ldg(sw + kb + 1);
        const uint32_t buf = n % C::kBufs;
        // the stage's scales came by TMA: wait on the stage itself before reading them
        ok = mbar_wait_bounded(&full[stage], phase, abort_flag, args.err, kPipelineTimeoutNs) &&
             mbar_wait_bounded(&tfull[buf], (n / C::kBufs) & 1, abort_flag, args.err, kPipelineTimeoutNs);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const float4 *s4 = reinterpret_cast<const float4 *>(sS + stage * kTok);
#pragma unroll
        for (int c = 0; c < kTok; c += 16) {
          uint32_t r[16];
          tmem_ld16(lanes + buf * kTok + c, r);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 s = s4[(c + i) / 4];
            acc[c + i] = fmaf(__uint_as_float(r[i]), s.x * w, acc[c + i]);
            acc[c + i + 1] = fmaf(__uint_as_float(r[i + 1]), s.y * w, acc[c + i + 1]);
            acc[c + i + 2] = fmaf(__uint_as_float(r[i + 2]), s.z * w, acc[c + i + 2]);
            acc[c + i + 3] = fmaf(__uint_as_float(r[i + 3]), s.w * w, acc[c + i + 3]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&tempty[buf]);
          mbar_arrive(&empty[stage]);
        }
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
      // the ring's last stage has been read by the MMAs (tfull) and no copy is in flight; the other
      // warps may still read scales, which lie behind the ring
#pragma unroll
      for (int j = 0; j < kTok; ++j) part[128 * j] = acc[j];
    } else {
      ok = mbar_wait_bounded(&tfull[0], 0, abort_flag, args.err, kPipelineTimeoutNs);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < 2 * kTok; c += 16) {
        uint32_t r[16];
        tmem_ld16(lanes + c, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) part[128 * (c + i)] = __uint_as_float(r[i]);
      }
    }
  }

  // ---------------------------------------------------------------- reduction over the ranks
  tc_fence_before();
  block_meet();
  if (splits > 1) cluster_meet();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, C::kTmemCols);
  if (*abort_flag == 0) {
    const int j0 = kTok * rank / splits, j1 = kTok * (rank + 1) / splits;
    const uint32_t base = smem_u32(smem);
    const int live = min(j1, args.M - m0);
    for (int e = static_cast<int>(threadIdx.x) + j0 * 128; e < live * 128; e += C::kThreads) {
      const int j = e >> 7, f = tile * 128 + (e & 127);
      float va[kStreamMaxSplit], vb[kStreamMaxSplit];  // every rank's load is in flight before the sums
#pragma unroll
      for (int r = 0; r < kStreamMaxSplit; ++r) {
        va[r] = vb[r] = 0.f;
        if (r < splits) {
          uint32_t at;
          asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(base + e * 4), "r"(r));
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(va[r]) : "r"(at) : "memory");
          if constexpr (!kFp8) asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(vb[r]) : "r"(at + kTok * 512) : "memory");
        }
      }
      float a = va[0], b = vb[0];
#pragma unroll
      for (int r = 1; r < kStreamMaxSplit; ++r)
        if (r < splits) {
          a += va[r];
          b += vb[r];
        }
      if (f < args.N) {
        const int64_t m = m0 + j;
        if constexpr (kFp8) {
          static_cast<uint16_t *>(args.out)[m * args.ldo + f] = T::one(a);
        } else {
          static_cast<uint16_t *>(args.out)[m * args.ldo + f] = T::one(act_fwd<kAct>(a) * b);
          if (args.save) {
            args.save[m * 2 * args.N + f] = a;
            args.save[m * 2 * args.N + args.N + f] = b;
          }
        }
      }
    }
  }
  if (splits > 1) cluster_meet();  // no CTA leaves while another reads its partial sums
}

template <bool kFp8, class T, int kAct, int kTok, bool kQuant = false>
cudaError_t launch_stream_gemm_as(const CUtensorMap &w0, const CUtensorMap &w1, const CUtensorMap &x,
                                  const StreamArgs &args, int splits, cudaStream_t s) {
  using C = StreamCfg<kFp8, kTok, kQuant>;
  auto kernel = stream_gemm_kernel<kFp8, T, kAct, kTok, kQuant>;
  static std::atomic<bool> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev].load()) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::kSmem));
    if (e != cudaSuccess) return e;
    ready[dev].store(true);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((args.N + 127) / 128 * splits),
                     static_cast<unsigned>((args.M + kTok - 1) / kTok));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, w0, w1, x, args, splits);
}

}  // namespace nvfp4
