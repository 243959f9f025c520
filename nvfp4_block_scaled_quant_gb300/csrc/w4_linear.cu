// Linear layer on 4-bit weights with group scales and 16-bit activations: the weights' preparation and the product of a
// few tokens, which is bound by the weights' bytes.
//
// A CTA takes one panel of 64 output features and a part of K (a cluster of `splits` CTAs shares a panel); its eight warps
// take the K blocks in turn.  Each warp has a ring of its own: lane 0 asks for the next block by one bulk copy
// as soon as the warp is done with the one in its place, so no warp waits for another until the sums are
// added up, over the warps and then over the cluster, in a fixed order (repeated calls give identical bits).
// The first blocks are asked for before the wait for the previous launch: prepared weights are final by then.
// One row with many outputs streams at 6.1 TB/s; small products are bound by the wait for the launch before, the first blocks'
// latency and the cluster's sums: 1 x 7168 -> 2048 4.6 us, 13 x 1536 -> 16384 7.3, 16 x 7168 -> 7168 13.6.
#include "w4.cuh"

namespace nvfp4 {
namespace {

// ---------------------------------------------------------------- preparation

// One block of prepared weights per CTA of 256 threads, 16 bytes of codes each.  Runs once, at load time.
__global__ void __launch_bounds__(256) w4_prepare_kernel(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros,
                                                         int64_t N, int64_t K, int64_t panels, int64_t blocks, int group,
                                                         bool gated, uint8_t *out, int block_bytes) {
  pdl_wait();  // no trigger: the next launch may read weights early
  const int64_t id = blockIdx.x, b = id % blocks, p = id / blocks % panels, m = id / blocks / panels;
  const int64_t n_groups = (K + group - 1) / group;
  uint8_t *dst = out + id * block_bytes;
  // the matrix row of a panel's row, -1 past its last
  auto row_of = [&](int r) -> int64_t {
    if (!gated) return p * kW4PanelRows + r < N ? p * kW4PanelRows + r : -1;
    const int64_t j = p * 32 + (r & 31);
    return j < N / 2 ? j + (r >= 32 ? N / 2 : 0) : -1;
  };
  const int tid = threadIdx.x, lane = tid & 31, pair = (tid >> 5) & 1, c = tid >> 6;
  const int64_t k = b * kW4BlockK + 32 * c + 8 * (lane & 3);
  uint32_t word[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = row_of(32 * pair + 8 * i + (lane >> 2));
    const uint32_t v = row >= 0 && k < K ? *reinterpret_cast<const uint32_t *>(codes + ((m * N + row) * K + k) / 2) : 0u;
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) w |= ((v >> (4 * e)) & 15u) << (16 * (e & 1) + 8 * ((e >> 1) & 1) + 4 * (e >> 2));
    word[i] = w;
  }
  reinterpret_cast<uint4 *>(dst)[tid] = make_uint4(word[0], word[1], word[2], word[3]);
  const int groups = kW4BlockK / group;
  if (tid < 64 * groups) {
    const int gi = tid >> 6, at = tid & 63;
    const int64_t row = row_of(16 * ((at >> 1) & 3) + 8 * (at & 1) + (at >> 3)), g = b * groups + gi;
    const bool live = row >= 0 && g < n_groups;
    reinterpret_cast<uint16_t *>(dst + kW4CodeBytes)[tid] = live ? scales[(m * N + row) * n_groups + g] : 0;
    if (zeros) dst[kW4CodeBytes + 128 * groups + tid] = live ? zeros[(m * N + row) * n_groups + g] & 15 : 0;
  }
}

// ---------------------------------------------------------------- few tokens

constexpr int kWarps = 8;

template <class T, int kGpb, bool kZeros, int kNT>
__global__ void __launch_bounds__(kWarps * 32, 2) w4_stream_kernel(const W4Args a, int splits, int depth) {
  constexpr int kBytes = w4_block_bytes(kGpb, kZeros);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kWarps][4];
  __shared__ int s_abort;
  volatile int *abort_flag = &s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = static_cast<int>(blockIdx.x) % splits, panel = static_cast<int>(blockIdx.x) / splits;
  const int tokens = a.M;  // at most 8 kNT
  const int blocks = (a.K + kW4BlockK - 1) / kW4BlockK;
  const int first = blocks * rank / splits, kb0 = first + warp, kb1 = blocks * (rank + 1) / splits;
  uint8_t *ring = smem + warp * depth * kBytes;
  const uint8_t *w = a.w + static_cast<int64_t>(panel) * blocks * kBytes;
  const uint64_t pol = policy_evict_normal();
  if (threadIdx.x == 0) s_abort = 0;
  if (lane == 0) {
    for (int s = 0; s < depth; ++s) mbar_init(&full[warp][s], 1);
    fence_barrier_init();
    for (int s = 0; s < depth && kb0 + s * kWarps < kb1; ++s) {
      mbar_arrive_expect_tx(&full[warp][s], kBytes);
      bulk_load(ring + s * kBytes, w + static_cast<int64_t>(kb0 + s * kWarps) * kBytes, kBytes, &full[warp][s], pol);
    }
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();

  uint64_t sums[4][kNT][2] = {};
  const uint16_t *x = static_cast<const uint16_t *>(a.x) + g * a.ldx + 8 * t;
  auto load_x = [&](int kb, W4Frag<kNT> &f) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        const int k = kb * kW4BlockK + 32 * c;
        f.v[c][n] = 8 * n + g < tokens && k + 8 * t < a.K
                        ? __ldg(reinterpret_cast<const uint4 *>(x + 8 * n * a.ldx + k))
                        : make_uint4(0u, 0u, 0u, 0u);
      }
  };
  bool ok = true;
  int stage = 0;
  uint32_t phase = 0;
  for (int kb = kb0; kb < kb1; kb += kWarps) {
    W4Frag<kNT> f;
    load_x(kb, f);
    ok = mbar_wait_bounded(&full[warp][stage], phase, abort_flag, a.err, kPipelineTimeoutNs);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    w4_block<T, kGpb, kZeros, kNT>(ring + stage * kBytes, f, sums);
    __syncwarp();
    if (lane == 0 && kb + depth * kWarps < kb1) {
      mbar_arrive_expect_tx(&full[warp][stage], kBytes);
      bulk_load(ring + stage * kBytes, w + static_cast<int64_t>(kb + depth * kWarps) * kBytes, kBytes, &full[warp][stage], pol);
    }
    if (++stage == depth) {
      stage = 0;
      phase ^= 1;
    }
  }
  if (!ok) {  // copies in flight land before the CTA's memory goes
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 10000000ull) {
    }
  }
  // the warp's ring is drained: its sums take its place
  w4_store_sums<kNT>(reinterpret_cast<float *>(ring), sums);
  __syncthreads();
  float *part = reinterpret_cast<float *>(smem);  // over warp 0's sums: each thread replaces what it alone reads
  const int pitch = depth * kBytes / 4;
  for (int e = threadIdx.x; e < tokens * kW4PanelRows; e += kWarps * 32) {
    const int at = (e >> 6) * kW4Pitch + (e & 63);
    float v = part[at];
#pragma unroll
    for (int u = 1; u < kWarps; ++u) v += part[u * pitch + at];
    part[at] = v * power_of_two(W4Scale<T>::kRest);
  }
  block_meet();
  if (splits > 1) cluster_meet();
  if (*abort_flag == 0) {
    const int live = tokens * kW4PanelRows, e0 = live * rank / splits, e1 = live * (rank + 1) / splits;
    const uint32_t base = smem_u32(smem);
    for (int e = e0 + static_cast<int>(threadIdx.x); e < e1; e += kWarps * 32) {
      const int at = (e >> 6) * kW4Pitch + (e & 63), n = panel * kW4PanelRows + (e & 63);
      const float s = cluster_sum(base + at * 4, splits);
      if (n < a.N) static_cast<uint16_t *>(a.y)[static_cast<int64_t>(e >> 6) * a.N + n] = T::one(s);
    }
  }
  if (splits > 1) cluster_meet();  // no CTA leaves while another reads its sums
}

template <class T, int kGpb, bool kZeros, int kNT>
cudaError_t stream_as(const W4Args &a, int splits, int depth, cudaStream_t s) {
  constexpr int kBytes = w4_block_bytes(kGpb, kZeros);
  const cudaError_t e = allow_smem<w4_stream_kernel<T, kGpb, kZeros, kNT>>(kWarps * 4 * kBytes);
  if (e != cudaSuccess) return e;
  return launch_clusters(w4_stream_kernel<T, kGpb, kZeros, kNT>, dim3(static_cast<unsigned>(w4_panels(a.N, false) * splits)), kWarps * 32,
                         static_cast<size_t>(kWarps) * depth * kBytes, splits, s, a, splits, depth);
}

template <class T, int kGpb, bool kZeros>
cudaError_t stream_tok(const W4Args &a, int tok8, int splits, int depth, cudaStream_t s) {
  return tok8 == 1 ? stream_as<T, kGpb, kZeros, 1>(a, splits, depth, s) : stream_as<T, kGpb, kZeros, 2>(a, splits, depth, s);
}
template <class T, int kGpb>
cudaError_t stream_zeros(const W4Args &a, bool zeros, int tok8, int splits, int depth, cudaStream_t s) {
  return zeros ? stream_tok<T, kGpb, true>(a, tok8, splits, depth, s) : stream_tok<T, kGpb, false>(a, tok8, splits, depth, s);
}
template <class T>
cudaError_t stream_group(const W4Args &a, int group, bool zeros, int tok8, int splits, int depth, cudaStream_t s) {
  if (group == 128) return stream_zeros<T, 1>(a, zeros, tok8, splits, depth, s);
  if (group == 64) return stream_zeros<T, 2>(a, zeros, tok8, splits, depth, s);
  return stream_zeros<T, 4>(a, zeros, tok8, splits, depth, s);
}

}  // namespace

cudaError_t launch_w4_prepare(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros, int64_t G, int64_t N,
                              int64_t K, int group, bool gated, uint8_t *out, cudaStream_t s) {
  const int64_t panels = w4_panels(N, gated), blocks = w4_blocks(K);
  return launch_pdl(w4_prepare_kernel, dim3(static_cast<unsigned>(G * panels * blocks)), dim3(256), 0, s, codes, scales, zeros,
                    N, K, panels, blocks, group, gated, out, w4_block_bytes(kW4BlockK / group, zeros != nullptr));
}

cudaError_t launch_w4_stream(const W4Args &a, int dtype, int group, bool zeros, int tok8, int splits, int depth,
                             cudaStream_t s) {
  return dtype == NVFP4_DT_BF16 ? stream_group<Bf16>(a, group, zeros, tok8, splits, depth, s)
                                : stream_group<Fp16>(a, group, zeros, tok8, splits, depth, s);
}

}  // namespace nvfp4
