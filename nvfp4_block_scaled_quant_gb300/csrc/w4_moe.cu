// A whole mixture-of-experts layer for a few tokens on 4-bit weights with group scales, in two kernels.
//
// 1. The router's logits x Wr^T, and zeroed counters for the second kernel.
// 2. Everything else.  Every CTA takes the top k of each token's logits itself and builds the same table of slots (an expert and
//    up to eight of its tokens); that costs less than a launch or a grid-wide exchange.  The work is a list of items in a
//    fixed order: first, slot by slot, panels of 32 gate and 32 up rows (h = act(g) u), then panels of 64 rows of
//    the down projection.  CTAs claim items one by one from a counter.  A down item waits until its slot's h
//    is complete; those items have lower numbers, so running CTAs hold them already, and however few CTAs run at
//    once, some claimed item can always go on.  While a CTA waits its producer warp goes on: the weights of the
//    next items stream into the ring regardless of h.
//    A slot's down rows go to the workspace in fp32; the CTA that finishes the last slot of a panel adds a token's experts
//    up in the order of its top k, so repeated calls give identical bits.
//
// With few tokens the layer is bound by the bytes of the chosen experts' weights.  Each block of 64 x 128 weights is
// one bulk copy into a ring of some 90 KB, two CTAs to an SM; eight warps split an item's K blocks and add their
// sums at its end.
#include <atomic>

#include "w4.cuh"

namespace nvfp4 {
namespace {

// ---------------------------------------------------------------- router logits

constexpr int kLogitWarps = 8;
constexpr int kLogitMaxSplit = 8;

// 16 experts per cluster, K split over its CTAs and their warps; kNT tiles of eight tokens.
template <class T, int kNT>
__global__ void __launch_bounds__(kLogitWarps * 32) w4_moe_logits_kernel(const W4MoeArgs a, int splits, int n_counters) {
  __shared__ float part[kLogitWarps][16 * 8 * kNT];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = static_cast<int>(blockIdx.x) % splits, tile = static_cast<int>(blockIdx.x) / splits;
  for (int i = blockIdx.x * (kLogitWarps * 32) + threadIdx.x; i < n_counters; i += gridDim.x * (kLogitWarps * 32)) a.counters[i] = 0;
  const int chunks = (a.H + 31) / 32, c0 = chunks * rank / splits, c1 = chunks * (rank + 1) / splits;
  const uint16_t *w = static_cast<const uint16_t *>(a.router) + static_cast<int64_t>(tile * 16 + g) * a.H + 8 * t;
  const uint16_t *x = static_cast<const uint16_t *>(a.x) + g * a.ldx + 8 * t;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  float acc[kNT][4] = {};
#pragma unroll(kNT == 1 ? 4 : 2)
  for (int c = c0 + warp; c < c1; c += kLogitWarps) {
    const int k = 32 * c;
    const bool in = k + 8 * t < a.H;
    const uint4 lo = in && tile * 16 + g < a.E ? __ldg(reinterpret_cast<const uint4 *>(w + k)) : zero;
    const uint4 hi = in && tile * 16 + g + 8 < a.E ? __ldg(reinterpret_cast<const uint4 *>(w + 8 * static_cast<int64_t>(a.H) + k)) : zero;
    const uint32_t a0[4] = {lo.x, hi.x, lo.y, hi.y}, a1[4] = {lo.z, hi.z, lo.w, hi.w};
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
      const uint4 b = in && 8 * n + g < a.T ? __ldg(reinterpret_cast<const uint4 *>(x + 8 * n * a.ldx + k)) : zero;
      mma16816<T>(acc[n], a0, b.x, b.y);
      mma16816<T>(acc[n], a1, b.z, b.w);
    }
  }
#pragma unroll
  for (int n = 0; n < kNT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) part[warp][(8 * n + 2 * t + (e & 1)) * 16 + 8 * (e >> 1) + g] = acc[n][e];
  __syncthreads();
  const int live = 16 * min(a.T, 8 * kNT);
  for (int e = threadIdx.x; e < live; e += kLogitWarps * 32) {
    float v = part[0][e];
#pragma unroll
    for (int u = 1; u < kLogitWarps; ++u) v += part[u][e];
    part[0][e] = v;
  }
  block_meet();
  if (splits > 1) cluster_meet();
  const uint32_t base = smem_u32(part);
  for (int e = live * rank / splits + static_cast<int>(threadIdx.x); e < live * (rank + 1) / splits; e += kLogitWarps * 32) {
    float v[kLogitMaxSplit];
#pragma unroll
    for (int r = 0; r < kLogitMaxSplit; ++r) {
      v[r] = 0.f;
      if (r < splits) {
        uint32_t addr;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(base + e * 4), "r"(r));
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[r]) : "r"(addr) : "memory");
      }
    }
    float s = v[0];
#pragma unroll
    for (int r = 1; r < kLogitMaxSplit; ++r)
      if (r < splits) s += v[r];
    const int expert = tile * 16 + (e & 15);
    if (expert < a.E) a.logits[static_cast<int64_t>(e >> 4) * a.E + expert] = s;
  }
  if (splits > 1) cluster_meet();
}

// ---------------------------------------------------------------- experts

constexpr int kWarps = 8, kThreads = (kWarps + 1) * 32;  // and a producer warp
constexpr int kItems = 4;                                // items known ahead
constexpr int kRedFloats = 8 * kW4Pitch;                 // a warp's sums: eight tokens
constexpr int kMaxStages = 24;

struct Plan {
  float weight[kW4MoeMaxEntries];      // of a token's chosen expert, entry t * topk + j
  uint16_t sorted[kW4MoeMaxEntries];   // entries ordered by expert
  uint16_t slot_expert[kW4MoeMaxSlots];
  uint16_t slot_first[kW4MoeMaxSlots]; // place of its first entry in `sorted` (shared expert: its first token)
  uint16_t slot_count[kW4MoeMaxSlots];
  int slots, shared_slots;
};
// While the plan is made, in the room of the sums: the experts' counts, first places and first slots, and the ids.
struct PlanScratch {
  int count[kW4MoeMaxExperts], first[kW4MoeMaxExperts], slot0[kW4MoeMaxExperts];
  uint16_t ids[kW4MoeMaxEntries];
};
static_assert(sizeof(PlanScratch) <= kWarps * kRedFloats * sizeof(float), "the scratch fits where the sums go");

// Order-preserving bits of a float (NaN above or below everything), never 0: 0 marks an expert that is taken.
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t b = __float_as_uint(v);
  const uint32_t k = b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
  return k ? k : 1u;
}

// The top k of one token's logits by a warp, the lowest expert first among equals; the weights are the softmax
// over all experts renormalised over the chosen ones, which is the softmax over the chosen ones.
template <int kPer>
__device__ __forceinline__ void top_k(const float *logits, int E, int topk, uint16_t *ids, float *weight) {
  const int lane = threadIdx.x & 31;
  uint32_t key[kPer];
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 32 * i;
    key[i] = e < E ? order_bits(__ldcg(logits + e)) : 0u;
    mine = max(mine, key[i]);
  }
  float first = 0.f, sum = 0.f, w = 0.f;
  for (int j = 0; j < topk; ++j) {
    const uint32_t best = __reduce_max_sync(0xffffffffu, mine);
    int at = 0x7fffffff;
    if (mine == best) {
#pragma unroll
      for (int i = kPer - 1; i >= 0; --i)
        if (key[i] == best) at = lane + 32 * i;
    }
    const int e = __reduce_min_sync(0xffffffffu, at);
    if (at == e) {  // taken: this lane's next best
      mine = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (lane + 32 * i == e) key[i] = 0u;
        mine = max(mine, key[i]);
      }
    }
    const float v = __uint_as_float(best ^ ((best >> 31) ? 0x80000000u : 0xFFFFFFFFu));
    if (j == 0) first = v;
    const float p = expf(v - first);
    sum += p;
    if (lane == j) {
      w = p;
      ids[j] = static_cast<uint16_t>(e);
    }
  }
  if (lane < topk) weight[lane] = __fdiv_rn(w, sum);
}

// The table of slots: the same in every CTA.
__device__ void make_plan(const W4MoeArgs &a, Plan &plan, PlanScratch &s) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, entries = a.T * a.topk;
  for (int e = tid; e < a.E; e += kThreads) s.count[e] = 0;
  for (int t = warp; t < a.T; t += kThreads / 32) {
    const float *l = a.logits + static_cast<int64_t>(t) * a.E;
    uint16_t *ids = s.ids + t * a.topk;
    float *w = plan.weight + t * a.topk;
    if (a.E <= 128)
      top_k<4>(l, a.E, a.topk, ids, w);
    else if (a.E <= 384)
      top_k<12>(l, a.E, a.topk, ids, w);
    else
      top_k<32>(l, a.E, a.topk, ids, w);
  }
  __syncthreads();
  for (int f = tid; f < entries; f += kThreads) atomicAdd(&s.count[s.ids[f]], 1);
  __syncthreads();
  const int shared_slots = a.sh13 ? (a.T + 7) / 8 : 0;
  if (warp == 0) {  // exclusive sums over the experts
    const int per = (a.E + 31) / 32, e0 = min(lane * per, a.E), e1 = min(e0 + per, a.E);
    int n = 0, slots = 0;
    for (int e = e0; e < e1; ++e) n += s.count[e], slots += (s.count[e] + 7) / 8;
    int n_at = n, slots_at = slots;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int u = __shfl_up_sync(0xffffffffu, n_at, o), v = __shfl_up_sync(0xffffffffu, slots_at, o);
      if (lane >= o) n_at += u, slots_at += v;
    }
    if (lane == 31) plan.slots = shared_slots + slots_at, plan.shared_slots = shared_slots;
    n_at -= n;
    slots_at += shared_slots - slots;
    for (int e = e0; e < e1; ++e) {
      s.first[e] = n_at, s.slot0[e] = slots_at;
      n_at += s.count[e], slots_at += (s.count[e] + 7) / 8;
    }
  }
  for (int i = tid; i < shared_slots; i += kThreads) {
    plan.slot_expert[i] = 0;
    plan.slot_first[i] = static_cast<uint16_t>(8 * i);
    plan.slot_count[i] = static_cast<uint16_t>(min(8, a.T - 8 * i));
  }
  __syncthreads();
  for (int f = tid; f < entries; f += kThreads) {
    const int e = s.ids[f];
    int rank = 0;  // entries of the same expert before this one
    for (int o = 0; o < f; ++o) rank += s.ids[o] == e;
    plan.sorted[s.first[e] + rank] = static_cast<uint16_t>(f);
    if (rank % 8 == 0) {
      const int slot = s.slot0[e] + rank / 8;
      plan.slot_expert[slot] = static_cast<uint16_t>(e);
      plan.slot_first[slot] = static_cast<uint16_t>(s.first[e] + rank);
      plan.slot_count[slot] = static_cast<uint16_t>(min(8, s.count[e] - rank));
    }
  }
  __syncthreads();
}

__device__ __forceinline__ int load_acquire(const int *p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void consumers_meet() {
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
}

__device__ __forceinline__ float activate(int act, float g) {
  if (act == NVFP4_ACT_SILU) return act_fwd<NVFP4_ACT_SILU>(g);
  if (act == NVFP4_ACT_GELU) return act_fwd<NVFP4_ACT_GELU>(g);
  return act_fwd<NVFP4_ACT_GELU_TANH>(g);
}

template <class T, int kGpb, bool kZeros>
__global__ void __launch_bounds__(kThreads, 2) w4_moe_experts_kernel(const W4MoeArgs a, int stages) {
  constexpr int kBytes = w4_block_bytes(kGpb, kZeros);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], item_full[kItems], item_empty[kItems];
  __shared__ int s_item[kItems], s_now, s_finish, s_abort;
  __shared__ Plan plan;
  volatile int *abort_flag = &s_abort;
  float *red = reinterpret_cast<float *>(smem + stages * kBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int q = 0; q < kItems; ++q) {
      mbar_init(&item_full[q], 1);
      mbar_init(&item_empty[q], 1);
    }
    s_abort = 0;
    s_finish = -1;
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  make_plan(a, plan, *reinterpret_cast<PlanScratch *>(red));

  const int slots = plan.slots, shared_slots = plan.shared_slots, entries = a.T * a.topk;
  const int panels13 = (a.I + 31) / 32, panels2 = (a.H + kW4PanelRows - 1) / kW4PanelRows;
  const int blocks13 = (a.H + kW4BlockK - 1) / kW4BlockK, blocks2 = (a.I + kW4BlockK - 1) / kW4BlockK;
  const int up_items = slots * panels13, items = up_items + slots * panels2;
  int *counter = a.counters, *slot_done = counter + kW4MoeCounters, *panel_done = slot_done + kW4MoeMaxSlots;

  if (warp == kWarps) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      const uint64_t pol = policy_evict_first();
      int stage = 0, q = 0;
      uint32_t phase = 0, qphase = 0;
      bool ok = true;
      int item = atomicAdd(counter, 1);
      for (;;) {
        ok = mbar_wait_bounded(&item_empty[q], qphase ^ 1, abort_flag, a.err, kPipelineTimeoutNs);
        if (!ok) break;
        s_item[q] = item < items ? item : -1;
        mbar_arrive(&item_full[q]);
        if (item >= items) break;
        const int next = atomicAdd(counter, 1);  // on its way while this item's blocks are asked for
        const bool up = item < up_items;
        const int i = up ? item : item - up_items, panels = up ? panels13 : panels2, blocks = up ? blocks13 : blocks2;
        const int slot = i / panels, panel = i - slot * panels;
        const uint8_t *w = slot < shared_slots ? (up ? a.sh13 : a.sh2) : (up ? a.w13 : a.w2);
        const int expert = plan.slot_expert[slot];
        w += (static_cast<int64_t>(expert) * panels + panel) * blocks * kBytes;
        for (int b = 0; b < blocks; ++b) {
          ok = mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, a.err, kPipelineTimeoutNs);
          if (!ok) break;
          mbar_arrive_expect_tx(&full[stage], kBytes);
          bulk_load(smem + stage * kBytes, w + static_cast<int64_t>(b) * kBytes, kBytes, &full[stage], pol);
          if (++stage == stages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if (++q == kItems) {
          q = 0;
          qphase ^= 1;
        }
        item = next;
      }
      if (!ok) {  // copies in flight land before the CTA's memory goes
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 10000000ull) {
        }
      }
    }
    return;
  }

  // ------------------------------------------------------------------ consumers
  const int g = lane >> 2, t = lane & 3;
  int q = 0;
  uint32_t qphase = 0;
  int stage0 = 0;  // stage and phase of the item's first block
  uint32_t phase0 = 0;
  for (;;) {
    if (tid == 0) {
      int item = -1;
      if (mbar_wait_bounded(&item_full[q], qphase, abort_flag, a.err, kPipelineTimeoutNs)) {
        item = s_item[q];
        mbar_arrive(&item_empty[q]);
        if (item >= up_items) {  // the slot's h is complete
          const int *done = slot_done + (item - up_items) / panels2;
          const uint64_t t0 = global_timer_ns();
          while (load_acquire(done) < panels13) {
            if (*abort_flag || global_timer_ns() - t0 > kPipelineTimeoutNs) {
              if (!*abort_flag) raise_device_error(a.err, NVFP4_DEVERR_PIPELINE_TIMEOUT);
              *abort_flag = 1;
              item = -1;
              break;
            }
          }
        }
      }
      s_now = item;
    }
    consumers_meet();
    const int item = s_now, finish = s_finish;
    if (finish >= 0) {
      // this CTA was the last to add to a panel of y: a token's experts in the order of its top k, then the shared one
      for (int e = tid; e < a.T * kW4PanelRows; e += kWarps * 32) {
        const int row = e >> 6, n = finish * kW4PanelRows + (e & 63);
        if (n < a.H) {
          const float *p = a.part + static_cast<int64_t>(row) * a.topk * a.H + n;
          float v = 0.f;
          for (int j = 0; j < a.topk; ++j) v = fmaf(plan.weight[row * a.topk + j], __ldcg(p + static_cast<int64_t>(j) * a.H), v);
          if (shared_slots) v += __ldcg(a.part + static_cast<int64_t>(entries + row) * a.H + n);
          static_cast<uint16_t *>(a.y)[static_cast<int64_t>(row) * a.H + n] = T::one(v);
        }
      }
    }
    if (item < 0) break;
    if (++q == kItems) {
      q = 0;
      qphase ^= 1;
    }
    const bool up = item < up_items;
    const int i = up ? item : item - up_items, panels = up ? panels13 : panels2, blocks = up ? blocks13 : blocks2;
    const int slot = i / panels, panel = i - slot * panels, count = plan.slot_count[slot], first = plan.slot_first[slot];
    const int width = up ? a.H : a.I;
    // the workspace row of the slot's token j, and this lane's activations
    auto row_of = [&](int j) { return slot < shared_slots ? entries + first + j : static_cast<int>(plan.sorted[first + j]); };
    const uint16_t *x = nullptr;
    if (g < count) {
      const int row = row_of(g);
      x = up ? static_cast<const uint16_t *>(a.x) + static_cast<int64_t>(row < entries ? row / a.topk : row - entries) * a.ldx
             : a.h + static_cast<int64_t>(row) * a.I;
      x += 8 * t;
    }
    auto load_x = [&](int b, W4Frag<1> &f) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int k = b * kW4BlockK + 32 * c;
        f.v[c][0] = x && k + 8 * t < width ? __ldcg(reinterpret_cast<const uint4 *>(x + k)) : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    float sums[4][1][4] = {};
    int stage = stage0 + warp;
    uint32_t phase = phase0;
    bool ok = true;
    for (int b = warp; b < blocks; b += kWarps) {
      W4Frag<1> f;
      load_x(b, f);
      while (stage >= stages) {
        stage -= stages;
        phase ^= 1;
      }
      ok = mbar_wait_bounded(&full[stage], phase, abort_flag, a.err, kPipelineTimeoutNs);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      w4_block<T, kGpb, kZeros, 1>(smem + stage * kBytes, f, sums);
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
      stage += kWarps;
    }
    stage0 += blocks;
    while (stage0 >= stages) {
      stage0 -= stages;
      phase0 ^= 1;
    }
    w4_store_sums<1>(red + warp * kRedFloats, sums);
    consumers_meet();
    if (up) {
      const int j = tid >> 5, c = tid & 31, n = panel * 32 + c;
      if (j < count && n < a.I) {
        float gate = 0.f, lift = 0.f;
#pragma unroll
        for (int u = 0; u < kWarps; ++u) {
          gate += red[u * kRedFloats + j * kW4Pitch + c];
          lift += red[u * kRedFloats + j * kW4Pitch + 32 + c];
        }
        a.h[static_cast<int64_t>(row_of(j)) * a.I + n] = T::one(activate(a.act, 16.f * gate) * (16.f * lift));
      }
    } else {
      for (int e = tid; e < count * kW4PanelRows; e += kWarps * 32) {
        const int j = e >> 6, n = panel * kW4PanelRows + (e & 63);
        float v = 0.f;
#pragma unroll
        for (int u = 0; u < kWarps; ++u) v += red[u * kRedFloats + j * kW4Pitch + (e & 63)];
        if (n < a.H) a.part[static_cast<int64_t>(row_of(j)) * a.H + n] = 16.f * v;
      }
    }
    consumers_meet();
    if (tid == 0) {  // the item's results are out
      __threadfence();
      int last = -1;
      if (up)
        atomicAdd(slot_done + slot, 1);
      else if (atomicAdd(panel_done + panel, 1) == slots - 1)
        last = panel;
      __threadfence();
      s_finish = last;
    }
  }
}

template <class T, int kNT>
cudaError_t logits_as(const W4MoeArgs &a, int splits, int n_counters, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.E + 15) / 16 * splits));
  cfg.blockDim = dim3(kLogitWarps * 32);
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
  return cudaLaunchKernelEx(&cfg, w4_moe_logits_kernel<T, kNT>, a, splits, n_counters);
}

template <class T, int kGpb, bool kZeros>
cudaError_t experts_as(const W4MoeArgs &a, int sms, cudaStream_t s) {
  constexpr int kBytes = w4_block_bytes(kGpb, kZeros);
  // two CTAs to an SM of 228 KB, of which each CTA's static part and 1 KB of the system's go off
  constexpr int kRed = kWarps * kRedFloats * 4, kStatic = 8192;
  constexpr int kFit = (233472 / 2 - 1024 - kStatic - kRed) / kBytes, kStages = kFit < kMaxStages ? kFit : kMaxStages;
  static_assert(kStages >= kWarps, "a stage for each warp");
  static_assert(sizeof(Plan) + (2 * kMaxStages + 2 * kItems) * 8 + 64 <= kStatic, "static shared memory");
  constexpr int kSmem = kStages * kBytes + kRed;
  auto kernel = w4_moe_experts_kernel<T, kGpb, kZeros>;
  static std::atomic<bool> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev].load()) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    ready[dev].store(true);
  }
  // no more CTAs than items
  const int64_t most = static_cast<int64_t>(a.T * a.topk + (a.sh13 ? (a.T + 7) / 8 : 0)) *
                       ((a.I + 31) / 32 + (a.H + kW4PanelRows - 1) / kW4PanelRows);
  const int64_t ctas = most < 2 * sms ? most : 2 * sms;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), kSmem, s, a, kStages);
}

template <class T>
cudaError_t moe_as(const W4MoeArgs &a, int group, bool zeros, int sms, cudaStream_t s) {
  const int tiles = (a.E + 15) / 16, chunks = (a.H + 31) / 32;
  int splits = sms / tiles;
  if (splits > chunks / kLogitWarps) splits = chunks / kLogitWarps;
  if (splits > kLogitMaxSplit) splits = kLogitMaxSplit;
  if (splits < 1) splits = 1;
  const int n = kW4MoeCounters + kW4MoeMaxSlots + (a.H + kW4PanelRows - 1) / kW4PanelRows;
  cudaError_t e = a.T <= 8 ? logits_as<T, 1>(a, splits, n, s) : a.T <= 16 ? logits_as<T, 2>(a, splits, n, s) : logits_as<T, 8>(a, splits, n, s);
  if (e != cudaSuccess) return e;
  if (group == 128) return zeros ? experts_as<T, 1, true>(a, sms, s) : experts_as<T, 1, false>(a, sms, s);
  if (group == 64) return zeros ? experts_as<T, 2, true>(a, sms, s) : experts_as<T, 2, false>(a, sms, s);
  return zeros ? experts_as<T, 4, true>(a, sms, s) : experts_as<T, 4, false>(a, sms, s);
}

}  // namespace

cudaError_t launch_w4_moe(const W4MoeArgs &a, int dtype, int group, bool zeros, int sms, cudaStream_t s) {
  return dtype == NVFP4_DT_BF16 ? moe_as<Bf16>(a, group, zeros, sms, s) : moe_as<Fp16>(a, group, zeros, sms, s);
}

}  // namespace nvfp4
