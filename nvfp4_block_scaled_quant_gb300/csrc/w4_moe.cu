// A whole mixture-of-experts layer for a few tokens on 4-bit weights with group scales, in two kernels.
//
// 1. The router's logits x Wr^T, and zeroed counters for the second kernel.
// 2. Everything else.  Every CTA takes the top k of each token's logits itself and builds the same table of slots (an expert and
//    up to eight of its tokens); that costs less than a launch or a grid-wide exchange.  The work is a list of items in a
//    fixed order: first, slot by slot, panels of 32 gate and 32 up rows (h = act(g) u), then panels of 64 rows of
//    the down projection, up to four panels to an item.  CTAs claim items one by one from a counter.  A down item waits until its slot's h
//    is complete; those items have lower numbers, so running CTAs hold them already, and however few CTAs run at
//    once, some claimed item can always go on.  While a CTA waits its producer warp goes on: the weights of the
//    next items stream into the ring regardless of h.
//    A slot's down rows go to the workspace in fp32; the CTA that finishes the last slot of a panel adds a token's experts
//    up in the order of its top k, so repeated calls give identical bits.
//
// h is held in 16 bits, the operand of the down product: one rounding of half a step, as in a layer that stores it; in 32 bits the
// product would take two operands.  In fp16 an h past 65504 would be an infinity where the layer's output need not be: a
// panel of such a row is stored times a power of two that brings its largest to 2^14, and the first warp that finds such a slot
// complete brings the other panels of the row to the same power.  Rows within the range are stored as they are.
//
// With few tokens the layer is bound by the bytes of the chosen experts' weights: 16 tokens, 384 experts of 7168 x 2048 390 us, 95% of
// the copy bandwidth; one token 50 us, of which 8 pass before weights stream.  Eight warps of a CTA share an item's
// panels and take a panel's K blocks in turn, each through a ring of its own: a block is one bulk copy.  A warp leaves its sums where its
// last block of the item was and goes on to the next item; a finishing warp adds the eight up and gives the
// stages back.  Two CTAs share an SM.  (The rings are the warps' own because a warp waits on every phase of its
// barriers then.  In a common ring, taken block by block, a warp that got a ring's length ahead of a slow copy would take an
// older phase of the same parity for its own.)
#include "w4.cuh"

namespace nvfp4 {
namespace {

// ---------------------------------------------------------------- router logits

constexpr int kLogitWarps = 8;

// 16 experts per cluster, K split over its CTAs and their warps; kNT tiles of eight tokens.  A chain of latencies (loads, sums over
// warps and cluster): 384 experts of 7168 and one token take about 5 us, 5.5 MB.
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
    const float s = cluster_sum(base + e * 4, splits);
    const int expert = tile * 16 + (e & 15);
    if (expert < a.E) a.logits[static_cast<int64_t>(e >> 4) * a.E + expert] = s;
  }
  if (splits > 1) cluster_meet();
}

// ---------------------------------------------------------------- experts

constexpr int kWarps = 8;                     // that multiply
constexpr int kThreads = (kWarps + 2) * 32;   // and a finishing and a producer warp
constexpr int kItems = 4;                     // items known ahead
constexpr int kMaxDepth = 3;                  // stages of a warp's ring

struct Plan {
  float weight[kW4MoeMaxEntries];      // of a token's chosen expert, entry t * topk + j
  uint16_t sorted[kW4MoeMaxEntries];   // entries ordered by expert
  uint16_t slot_expert[kW4MoeMaxSlots];
  uint16_t slot_first[kW4MoeMaxSlots]; // place of its first entry in `sorted` (shared expert: its first token)
  uint16_t slot_count[kW4MoeMaxSlots];
  int slots, shared_slots;
};
// While the plan is made, in the room of the rings: each expert's tokens as a bit mask, the place of its first entry and its first
// slot (16 bits each), and the ids.
struct PlanScratch {
  uint32_t tokens[2][kW4MoeMaxExperts + 32], first[kW4MoeMaxExperts + 32];
  uint16_t ids[kW4MoeMaxEntries];
};
// An expert's place there, such that lanes that read 32 experts apart meet different banks.
__device__ __forceinline__ int spread(int e) { return e + (e >> 5); }
static_assert(kW4MoeMaxT <= 64, "a token is a bit of two words");
// Order-preserving bits of a float (NaN above or below everything), never 0: 0 marks an expert that is taken.
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t b = __float_as_uint(v);
  const uint32_t k = b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
  return k ? k : 1u;
}
__device__ __forceinline__ float order_value(uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu)); }

// The top k of one token's logits by a warp, the lowest expert first among equals; the weights are the softmax
// over all experts renormalised over the chosen ones, which is the softmax over the chosen ones.  A lane holds every 32nd
// logit and knows its best two.  The rounds are one after the other: each takes the best of all, whose lane goes on to its
// second, or looks for the next one in the rare case that it has given that up too (looking every time took 400 cycles a
// round at 384 experts).
template <int kPer>
__device__ __forceinline__ void top_k(const uint32_t (&key)[kPer], int topk, uint16_t *ids, float *weight) {
  const int lane = threadIdx.x & 31;
  uint32_t best = 0, second = 0;
  int at = 0, at2 = 0;  // their places, the first among equals
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (key[i] > best)
      second = best, at2 = at, best = key[i], at = i;
    else if (key[i] > second)
      second = key[i], at2 = i;
  }
  float mine = -INFINITY;  // lane j: the logit of the j-th choice
  for (int j = 0; j < topk; ++j) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const uint32_t holders = __ballot_sync(0xffffffffu, best == top);
    bool taken = best == top;
    if (holders & (holders - 1)) {  // several lanes: the lowest expert's
      const int e = __reduce_min_sync(0xffffffffu, taken ? lane + 32 * at : 0x7fffffff);
      taken = (e & 31) == lane;
    }
    if (lane == j) mine = order_value(top);
    if (taken) {
      ids[j] = static_cast<uint16_t>(lane + 32 * at);
      if (second) {
        best = second, at = at2, second = 0;
      } else {  // the next behind this one
        uint32_t next = 0;
        int next_at = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if ((key[i] < best || (key[i] == best && i > at)) && key[i] > next) next = key[i], next_at = i;
        best = next, at = next_at;
      }
    }
  }
  const float first = __shfl_sync(0xffffffffu, mine, 0);
  const float p = lane < topk ? expf(mine - first) : 0.f;
  float sum = p;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane < topk) weight[lane] = __fdiv_rn(p, sum);
}

// ... of this warp's tokens, the next one's logits on their way meanwhile.
template <int kPer>
__device__ __forceinline__ void choose(const W4MoeArgs &a, uint16_t *ids, float *weight) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t next[kPer];
  auto load = [&](int t) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) next[i] = lane + 32 * i < a.E ? __float_as_uint(__ldcg(a.logits + t * a.E + lane + 32 * i)) : 0u;
  };
  if (warp < a.T) load(warp);
  for (int t = warp; t < a.T; t += kThreads / 32) {
    uint32_t key[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) key[i] = lane + 32 * i < a.E ? order_bits(__uint_as_float(next[i])) : 0u;
    if (t + kThreads / 32 < a.T) load(t + kThreads / 32);
    top_k<kPer>(key, a.topk, ids + t * a.topk, weight + t * a.topk);
  }
}

// How many panels (log2) an item holds, shared out to the warps, so that a warp has more K blocks in a row and the items' own
// cost (the first load of its activations, its sums, its signals) is spread over more of them.  That pays where a CTA takes many items; where it
// takes few, smaller ones spread better.  Two panels / one: 59 tokens, 80 experts of 5280 x 352 (22 items of the down projection to a
// CTA) 98 / 110 us, 32 tokens, 180 of 1256 x 1808 (26 and 9) 112 / 125; 1 token, 384 of 7168 x 2048 (2 and 3) 54 / 50.
__device__ __forceinline__ int item_split(int slots, int panels, int ctas) {
  const int rounds = slots * panels / ctas;
  return rounds < 8 ? 0 : rounds < 32 ? 1 : 2;
}

// The table of slots, the same in every CTA: experts in their order, tokens in theirs.
__device__ void make_plan(const W4MoeArgs &a, Plan &plan, PlanScratch &s) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, entries = a.T * a.topk;
  if (entries > 32)
    for (int e = tid; e < a.E; e += kThreads) s.tokens[0][spread(e)] = s.tokens[1][spread(e)] = 0u;
  // (with four places to a lane, where it has one expert, each choice ends in a search: 53 tokens, 28 experts, top 8 37 us instead of 30)
  if (a.E <= 32)
    choose<1>(a, s.ids, plan.weight);
  else if (a.E <= 128)
    choose<4>(a, s.ids, plan.weight);
  else if (a.E <= 384)
    choose<12>(a, s.ids, plan.weight);
  else
    choose<32>(a, s.ids, plan.weight);
  const int shared_slots = a.sh13 ? (a.T + 7) / 8 : 0;
  for (int i = tid; i < shared_slots; i += kThreads) {
    plan.slot_expert[i] = 0;
    plan.slot_first[i] = static_cast<uint16_t>(8 * i);
    plan.slot_count[i] = static_cast<uint16_t>(min(8, a.T - 8 * i));
  }
  __syncthreads();
  if (entries <= 32) {
    // few entries: a warp counts the ones of smaller experts and the earlier ones of the same expert
    if (warp == 0) {
      const int e = lane < entries ? s.ids[lane] : 0x7fff;
      int rank = 0, same = 0, less = 0, slot = shared_slots;
      for (int o = 0; o < entries; ++o) {
        const int u = __shfl_sync(0xffffffffu, e, o);
        rank += u == e && o < lane, same += u == e, less += u < e;
      }
      const uint32_t heads = __ballot_sync(0xffffffffu, lane < entries && rank % 8 == 0);
      for (int o = 0; o < entries; ++o) slot += __shfl_sync(0xffffffffu, e, o) < e && (heads >> o & 1);
      if (lane < entries) {
        plan.sorted[less + rank] = static_cast<uint16_t>(lane);
        if (rank % 8 == 0) {
          plan.slot_expert[slot + rank / 8] = static_cast<uint16_t>(e);
          plan.slot_first[slot + rank / 8] = static_cast<uint16_t>(less + rank);
          plan.slot_count[slot + rank / 8] = static_cast<uint16_t>(min(8, same - rank));
        }
      }
      if (lane == 0) plan.slots = shared_slots + __popc(heads), plan.shared_slots = shared_slots;
    }
    __syncthreads();
    return;
  }
  for (int f = tid; f < entries; f += kThreads) {
    const int t = f / a.topk;
    atomicOr(&s.tokens[t >> 5][spread(s.ids[f])], 1u << (t & 31));
  }
  __syncthreads();
  // exclusive sums over the experts, entries in the low and slots in the high half: each lane of a warp those of `per`
  // experts in a row, twice
  if (warp == 0) {
    const int per = (a.E + 31) / 32, e0 = lane * per, e1 = min(e0 + per, a.E);
    uint32_t own = 0;
    auto both = [&](int e) {
      const uint32_t n = __popc(s.tokens[0][spread(e)]) + __popc(s.tokens[1][spread(e)]);
      return n | ((n + 7) / 8 << 16);
    };
    for (int e = e0; e < e1; ++e) own += both(e);
    uint32_t sum = own;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += u;
    }
    if (lane == 31) plan.slots = shared_slots + static_cast<int>(sum >> 16), plan.shared_slots = shared_slots;
    sum += (static_cast<uint32_t>(shared_slots) << 16) - own;
    for (int e = e0; e < e1; ++e) {
      s.first[spread(e)] = sum;
      sum += both(e);
    }
  }
  __syncthreads();
  for (int f = tid; f < entries; f += kThreads) {
    const int e = s.ids[f], t = f / a.topk;
    const uint32_t m0 = s.tokens[0][spread(e)], m1 = s.tokens[1][spread(e)], below = (1u << (t & 31)) - 1u;
    const int n = __popc(m0) + __popc(m1), rank = t < 32 ? __popc(m0 & below) : __popc(m0) + __popc(m1 & below);
    const uint32_t start = s.first[spread(e)];
    const int first = static_cast<int>(start & 0xFFFFu) + rank;
    plan.sorted[first] = static_cast<uint16_t>(f);
    if (rank % 8 == 0) {
      const int slot = static_cast<int>(start >> 16) + rank / 8;
      plan.slot_expert[slot] = static_cast<uint16_t>(e);
      plan.slot_first[slot] = static_cast<uint16_t>(first);
      plan.slot_count[slot] = static_cast<uint16_t>(min(8, n - rank));
    }
  }
  __syncthreads();
}

__device__ __forceinline__ int load_acquire(const int *p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float activate(int act, float g) {
  if (act == NVFP4_ACT_SILU) return act_fwd<NVFP4_ACT_SILU>(g);
  if (act == NVFP4_ACT_GELU) return act_fwd<NVFP4_ACT_GELU>(g);
  return act_fwd<NVFP4_ACT_GELU_TANH>(g);
}

// The workspace row of a slot's token j.
__device__ __forceinline__ int slot_row(const Plan &plan, int entries, int slot, int j) {
  const int at = plan.slot_first[slot] + j;
  return slot < plan.shared_slots ? entries + at : static_cast<int>(plan.sorted[at]);
}

// fp16: a slot's count has its finished items in the low bits and counts those with panels past the type's range from kSlotWide on.
// A warp that finds the count complete and such panels in it comes here: the first brings every panel of such a row to the row's
// largest power, the others wait.
constexpr int kSlotWide = 1 << 10, kSlotClaimed = 1 << 28, kSlotSettled = 1 << 29;
static_assert(kW4MoeMaxDim / 32 < kSlotWide && kW4MoeMaxDim / 32 * kSlotWide < kSlotClaimed, "items of a slot");
__device__ __noinline__ bool settle(uint16_t *h, int I, const uint8_t *powers, int64_t ld_powers, const int *row_power, const Plan &plan, int entries,
                                    int slot, int *done, volatile int *abort_flag, uint32_t *err) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
  int before = 0;
  if (lane == 0) before = atomicOr(done, kSlotClaimed);
  before = __shfl_sync(0xffffffffu, before, 0);
  if (before & kSlotClaimed) {
    bool ok = true;
    const uint64_t t0 = global_timer_ns();
    while (!(load_acquire(done) & kSlotSettled)) {
      if (*abort_flag || global_timer_ns() - t0 > kPipelineTimeoutNs) {
        if (!*abort_flag) raise_device_error(err, NVFP4_DEVERR_PIPELINE_TIMEOUT);
        *abort_flag = 1;
        ok = false;
        break;
      }
    }
    return __all_sync(0xffffffffu, ok) != 0;
  }
  __threadfence();  // behind the panels, whose counts were seen
  for (int j = 0; j < plan.slot_count[slot]; ++j) {
    const int row = slot_row(plan, entries, slot, j), most = __ldcg(row_power + row);
    if (most == 0) continue;
    uint32_t *pairs = reinterpret_cast<uint32_t *>(h + static_cast<int64_t>(row) * I);
    for (int i = lane; i < I / 2; i += 32) {
      const float f = power_of_two(__ldcg(powers + row * ld_powers + i / 16) - most);
      const uint32_t v = __ldcg(pairs + i);
      pairs[i] = Fp16::pack(Fp16::lo(v) * f, Fp16::hi(v) * f);
    }
  }
  __threadfence();
  __syncwarp();
  if (lane == 0) atomicOr(done, kSlotSettled);
  return true;
}

// An item of the list.
struct Item {
  int slot;  // -1: no more items
  int panel, blocks, up;  // its first panel
};

template <class T, int kGpb, bool kZeros>
__global__ void __launch_bounds__(kThreads, 2) w4_moe_experts_kernel(const W4MoeArgs a, const int most) {
  constexpr int kBytes = w4_block_bytes(kGpb, kZeros);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kWarps][kMaxDepth], empty[kWarps][kMaxDepth], item_full[kItems], item_empty[kItems], sums_full[2], sums_empty[2];
  __shared__ int4 s_item[kItems];
  __shared__ int s_sums[2][kWarps], s_finished, s_abort;
  __shared__ uint16_t s_panels[kW4MoeMaxDim / kW4PanelRows];  // of y, that this CTA finishes
  __shared__ Plan plan;
  volatile int *abort_flag = &s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int w = 0; w < kWarps; ++w)
      for (int s = 0; s < most; ++s) {
        mbar_init(&full[w][s], 1);
        mbar_init(&empty[w][s], 1);
      }
    for (int q = 0; q < kItems; ++q) {
      mbar_init(&item_full[q], 1);
      mbar_init(&item_empty[q], kWarps + 1);
    }
    for (int u = 0; u < 2; ++u) {
      mbar_init(&sums_full[u], kWarps);
      mbar_init(&sums_empty[u], 1);
    }
    s_abort = 0;
    s_finished = 0;
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  // the first item, on its way while the plan is made
  int first_item = 0;
  if (tid == (kWarps + 1) * 32) first_item = atomicAdd(a.counters, 1);
  make_plan(a, plan, *reinterpret_cast<PlanScratch *>(smem));

  const int slots = plan.slots, shared_slots = plan.shared_slots, entries = a.T * a.topk;
  const int panels13 = (a.I + 31) / 32, panels2 = (a.H + kW4PanelRows - 1) / kW4PanelRows;
  const int blocks13 = (a.H + kW4BlockK - 1) / kW4BlockK, blocks2 = (a.I + kW4BlockK - 1) / kW4BlockK;
  const int split13 = item_split(slots, panels13, gridDim.x), split2 = item_split(slots, panels2, gridDim.x);
  const int items13 = (panels13 + (1 << split13) - 1) >> split13, items2 = (panels2 + (1 << split2) - 1) >> split2;  // of a slot
  // Stages of a warp's ring.  The producer claims an item a ring ahead of the products, which with few items leaves some to a CTA that
  // is behind while others run out: two stages where items are few and small, else three.  Three / two: one token 51.3 /
  // 49.7 us, 13 tokens, 24 experts of 1544 x 1000 36 / 34, 16 tokens, 384 of 7168 x 2048 390 / 402.
  const int depth = split2 == 0 ? 2 : most;
  int *counter = a.counters, *slot_done = counter + kW4MoeSlotDone, *row_power = counter + kW4MoeRowPower, *panel_done = counter + kW4MoeCounters;
  constexpr bool kPowers = T::kCode == NVFP4_DT_FP16;  // h may pass the type's range
  auto row_of = [&](int slot, int j) { return slot_row(plan, entries, slot, j); };

  if (warp == kWarps + 1) {
    // ---------------------------------------------------------------- producer: lane w fills the ring of warp w
    const int up_items = slots * items13, items = up_items + slots * items2;
    const uint64_t pol = policy_evict_first();
    fence_proxy_async_shared();  // the plan's scratch was where the copies go
    int stage = 0, q = 0;
    uint32_t phase = 0, qphase = 0;
    bool ok = true;
    int item = first_item;
    for (;;) {
      item = __shfl_sync(0xffffffffu, item, 0);
      const bool up = item < up_items;
      const int i = up ? item : item - up_items, n = up ? items13 : items2, blocks = up ? blocks13 : blocks2;
      const int slot = item < items ? i / n : -1, panel0 = i % n << (up ? split13 : split2);
      if (lane == 0) {
        ok = mbar_wait_bounded(&item_empty[q], qphase ^ 1, abort_flag, a.err, kPipelineTimeoutNs);
        s_item[q] = make_int4(slot, panel0, blocks, up);
        if (ok) mbar_arrive(&item_full[q]);
      }
      if (++q == kItems) {
        q = 0;
        qphase ^= 1;
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok || slot < 0) break;
      if (lane == 0) item = atomicAdd(counter, 1);  // the next one, on its way while this one's blocks are asked for
      const uint8_t *w = slot < shared_slots ? (up ? a.sh13 : a.sh2) : (up ? a.w13 : a.w2);
      const int warps = kWarps >> (up ? split13 : split2), panels = up ? panels13 : panels2, panel = panel0 + lane / warps;
      w += (static_cast<int64_t>(plan.slot_expert[slot]) * panels + panel) * blocks * kBytes;
      if (lane < kWarps && panel < panels) {
        for (int b = lane % warps; b < blocks; b += warps) {
          ok = mbar_wait_bounded(&empty[lane][stage], phase ^ 1, abort_flag, a.err, kPipelineTimeoutNs);
          if (!ok) break;
          mbar_arrive_expect_tx(&full[lane][stage], kBytes);
          bulk_load(smem + (lane * depth + stage) * kBytes, w + static_cast<int64_t>(b) * kBytes, kBytes, &full[lane][stage], pol);
          if (++stage == depth) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // no lane begins an item before every block of the one before it is asked for
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
    }
    if (!ok) {  // copies in flight land before the CTA's memory goes
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 10000000ull) {
      }
    }
    return;
  }

  // the next item of the queue for a whole warp; slot -1 behind the last one or after a wait that gave up
  int q = 0;
  uint32_t qphase = 0;
  auto next_item = [&] {
    const bool ok = mbar_wait_bounded(&item_full[q], qphase, abort_flag, a.err, kPipelineTimeoutNs);
    const int4 v = s_item[q];
    const Item item = {__all_sync(0xffffffffu, ok) ? v.x : -1, v.y, v.z, v.w};
    __syncwarp();
    if (lane == 0 && ok) mbar_arrive(&item_empty[q]);
    if (++q == kItems) {
      q = 0;
      qphase ^= 1;
    }
    return item;
  };

  if (warp < kWarps) {
    // ---------------------------------------------------------------- products
    const int g = lane >> 2, t = lane & 3;
    const uint8_t *ring = smem + warp * depth * kBytes;
    const uint32_t topk_inverse = (65536u + a.topk - 1) / a.topk;  // entries are below 512, topk at most 16: exact
    int stage = 0, buf = 0;
    uint32_t phase = 0, bphase = 0;
    int ready = -1;  // the last slot whose h was seen complete
    Item item = next_item();
    // This lane's activations of the item.  Lanes of tokens that the slot does not have take its first one's: their columns
    // of the sums are left where they are.
    const uint16_t *x = nullptr;
    int width = 0;
    auto open = [&](const Item &it) {
      width = it.up ? a.H : a.I;
      const int row = row_of(it.slot, g < plan.slot_count[it.slot] ? g : 0);
      const int token = row < entries ? static_cast<int>((row * topk_inverse) >> 16) : row - entries;
      x = it.up ? static_cast<const uint16_t *>(a.x) + token * a.ldx : a.h + static_cast<int64_t>(row) * a.I;
      x += 8 * t;
    };
    auto load_x = [&](int b, W4Frag<1> &f) {
      const uint16_t *p = x + b * kW4BlockK;
      if ((b + 1) * kW4BlockK <= width) {
#pragma unroll
        for (int c = 0; c < 4; ++c) f.v[c][0] = __ldcg(reinterpret_cast<const uint4 *>(p + 32 * c));
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          f.v[c][0] = b * kW4BlockK + 32 * c + 8 * t < width ? __ldcg(reinterpret_cast<const uint4 *>(p + 32 * c)) : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    bool ok = true;
    while (item.slot >= 0) {
      const Item it = item;
      if (!it.up && ready != it.slot) {  // its h is complete
        const uint64_t t0 = global_timer_ns();
        int seen;
        while (((seen = load_acquire(slot_done + it.slot)) & (kSlotWide - 1)) < items13) {
          if (*abort_flag || global_timer_ns() - t0 > kPipelineTimeoutNs) {
            if (!*abort_flag) raise_device_error(a.err, NVFP4_DEVERR_PIPELINE_TIMEOUT);
            *abort_flag = 1;
            ok = false;
            break;
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (kPowers && ok && __any_sync(0xffffffffu, seen >= kSlotWide))
          ok = settle(a.h, a.I, a.powers, a.ld_powers, row_power, plan, entries, it.slot, slot_done + it.slot, abort_flag, a.err);
        if (!ok) break;
        ready = it.slot;
      }
      open(it);
      // this warp's panel of the item, and its K blocks: every `warps`-th from the first
      const int shift = it.up ? split13 : split2, warps = kWarps >> shift, first = warp & (warps - 1);
      const bool some = it.panel + (warp >> (3 - shift)) < (it.up ? panels13 : panels2) && first < it.blocks;
      uint64_t sums[4][1][2] = {};
      for (int b = first; some && b < it.blocks; b += warps) {
        W4Frag<1> f;
        load_x(b, f);
        ok = mbar_wait_bounded(&full[warp][stage], phase, abort_flag, a.err, kPipelineTimeoutNs);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        w4_block<T, kGpb, kZeros, 1>(ring + stage * kBytes, f, sums);
        __syncwarp();
        if (b + warps >= it.blocks) break;  // the item's sums go where its last block was
        if (lane == 0) mbar_arrive(&empty[warp][stage]);
        if (++stage == depth) {
          stage = 0;
          phase ^= 1;
        }
      }
      ok = ok && mbar_wait_bounded(&sums_empty[buf], bphase ^ 1, abort_flag, a.err, kPipelineTimeoutNs);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (some) {
        w4_store_sums<1>(reinterpret_cast<float *>(smem + (warp * depth + stage) * kBytes), sums);
        fence_proxy_async_shared();  // a copy takes their place later
        if (lane == 0) s_sums[buf][warp] = stage;
        if (++stage == depth) {
          stage = 0;
          phase ^= 1;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sums_full[buf]);
      if (++buf == 2) {
        buf = 0;
        bphase ^= 1;
      }
      item = next_item();
    }
  } else {
    // ---------------------------------------------------------------- finishing warp: an item's sums over the warps
    const float kUnscale = power_of_two(W4Scale<T>::kRest);
    int buf = 0, finished = 0, rows_slot = -1, rows_up = 0, row = 0;
    float unscale = 0.f;
    uint32_t bphase = 0;
    for (;;) {
      const Item it = next_item();
      if (it.slot < 0) break;
      bool ok = mbar_wait_bounded(&sums_full[buf], bphase, abort_flag, a.err, kPipelineTimeoutNs);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const int count = plan.slot_count[it.slot], shift = it.up ? split13 : split2, warps = kWarps >> shift;
      const int parts = min(it.blocks, warps), panels = min(1 << shift, (it.up ? panels13 : panels2) - it.panel);
      if (it.slot != rows_slot || it.up != rows_up) {  // lane j: the workspace row of token j, and the factor of its sums of the down product
        rows_slot = it.slot, rows_up = it.up;
        row = row_of(it.slot, min(lane & 7, count - 1));
        if (kPowers && !it.up) unscale = power_of_two(W4Scale<T>::kRest + __ldcg(row_power + row));
      }
      const float *r[kWarps];
#pragma unroll
      for (int u = 0; u < kWarps; ++u) r[u] = reinterpret_cast<const float *>(smem + (u * depth + s_sums[buf][u]) * kBytes);
      auto sum4 = [&](uint32_t in, int at) {  // over the warps of `in`, in their order
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int u = 0; u < kWarps; ++u)
          if (in >> u & 1) {
            const float4 p = *reinterpret_cast<const float4 *>(r[u] + at);
            v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
          }
        return v;
      };
      bool wide = false;  // a row's panel passed the type's range
      for (int sub = 0; sub < panels; ++sub) {
        const uint32_t in = ((1u << parts) - 1u) << (sub * warps);  // the warps that hold its sums
        if (it.up) {
          // four tokens at a time, four outputs to a lane
          const int c = 4 * (lane & 7), n = (it.panel + sub) * 32 + c;
          for (int j0 = 0; j0 < count; j0 += 4) {
            const int j = j0 + (lane >> 3), to = __shfl_sync(0xffffffffu, row, j & 7);
            const bool live = j < count && n < a.I;
            float v[4] = {}, largest = 0.f;
            if (live) {
              const float4 gate = sum4(in, j * kW4Pitch + c), lift = sum4(in, j * kW4Pitch + 32 + c);
              auto out = [&](float gv, float lv) { return activate(a.act, gv * kUnscale) * (lv * kUnscale); };
              v[0] = out(gate.x, lift.x), v[1] = out(gate.y, lift.y), v[2] = out(gate.z, lift.z), v[3] = out(gate.w, lift.w);
            }
            if constexpr (kPowers) {
#pragma unroll
              for (int i = 0; i < 4; ++i) largest = fmaxf(largest, fabsf(v[i]));
#pragma unroll
              for (int o = 4; o; o >>= 1) largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, o));
              const int bits = __float_as_int(largest), power = largest > 65504.f && bits < 0x7F800000 ? (bits >> 23) - 127 - 14 : 0;
              wide |= __any_sync(0xffffffffu, power) != 0;
              if (power) {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] *= power_of_two(-power);
              }
              if (live && c == 0) {
                a.powers[to * a.ld_powers + it.panel + sub] = static_cast<uint8_t>(power);
                if (power) atomicMax(row_power + to, power);
              }
            }
            if (live)
              *reinterpret_cast<uint2 *>(a.h + static_cast<int64_t>(to) * a.I + n) = make_uint2(T::pack(v[0], v[1]), T::pack(v[2], v[3]));
          }
        } else {
          // two tokens at a time, four outputs to a lane
          const int c = 4 * (lane & 15), n = (it.panel + sub) * kW4PanelRows + c;
          for (int j0 = 0; j0 < count; j0 += 2) {
            const int j = j0 + (lane >> 4), to = __shfl_sync(0xffffffffu, row, j & 7);
            const float u = kPowers ? __shfl_sync(0xffffffffu, unscale, j & 7) : kUnscale;
            if (j < count && n < a.H) {
              const float4 v = sum4(in, j * kW4Pitch + c);
              *reinterpret_cast<float4 *>(a.part + static_cast<int64_t>(to) * a.H + n) = make_float4(v.x * u, v.y * u, v.z * u, v.w * u);
            }
          }
        }
      }
      // the stages go back to the copies
      fence_proxy_async_shared();
      __syncwarp();
      if (lane < panels * warps && (lane & (warps - 1)) < parts) mbar_arrive(&empty[lane][s_sums[buf][lane]]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sums_empty[buf]);
      __threadfence();  // the item's results are out
      __syncwarp();
      if (it.up) {
        if (lane == 0) atomicAdd(slot_done + it.slot, wide ? kSlotWide + 1 : 1);
      } else {
        const bool last = lane < panels && atomicAdd(panel_done + it.panel + lane, 1) == slots - 1;
        const uint32_t ends = __ballot_sync(0xffffffffu, last);
        if (last) s_panels[finished + __popc(ends & ((1u << lane) - 1u))] = static_cast<uint16_t>(it.panel + lane);
        finished += __popc(ends);
      }
      if (++buf == 2) {
        buf = 0;
        bphase ^= 1;
      }
    }
    __threadfence();  // behind the counts that were seen full
    if (lane == 0) s_finished = finished;
  }
  // Panels of y to which this CTA was the last to add: a token's experts in the order of its top k, then the shared one.
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"((kWarps + 1) * 32) : "memory");
  // Two or four columns to a thread: four are fewer turns where a panel has more than a pair for each thread (51 tokens, 116
  // experts of 1384 x 184 56.6 -> 51.8 us), two 1% less time where it has not.
  const int finished_rows = s_finished * a.T;
  auto add_up = [&](auto pair) {
    using V = decltype(pair);
    constexpr int kCols = sizeof(V) / 4, kChunks = kW4PanelRows / kCols;
    for (int e = tid; e < finished_rows * kChunks; e += (kWarps + 1) * 32) {
      const int at = e / kChunks, row = at % a.T, n = s_panels[at / a.T] * kW4PanelRows + kCols * (e % kChunks);
      if (n >= a.H) continue;
      const float *p = a.part + static_cast<int64_t>(row) * a.topk * a.H + n;
      V u[9];
      float v[kCols] = {};
      for (int j0 = 0; j0 < a.topk; j0 += 8) {  // eight loads and the shared expert's in flight
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j0 + j < a.topk) u[j] = __ldcg(reinterpret_cast<const V *>(p + static_cast<int64_t>(j0 + j) * a.H));
        if (shared_slots && j0 + 8 >= a.topk) u[8] = __ldcg(reinterpret_cast<const V *>(a.part + static_cast<int64_t>(entries + row) * a.H + n));
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j0 + j < a.topk) {
            const float w = plan.weight[row * a.topk + j0 + j];
#pragma unroll
            for (int c = 0; c < kCols; ++c) v[c] = fmaf(w, reinterpret_cast<const float *>(&u[j])[c], v[c]);
          }
      }
      if (shared_slots) {
#pragma unroll
        for (int c = 0; c < kCols; ++c) v[c] += reinterpret_cast<const float *>(&u[8])[c];
      }
      uint32_t *y = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.y) + static_cast<int64_t>(row) * a.H + n);
      if constexpr (kCols == 4)
        *reinterpret_cast<uint2 *>(y) = make_uint2(T::pack(v[0], v[1]), T::pack(v[2], v[3]));
      else
        *y = T::pack(v[0], v[1]);
    }
  };
  if (a.T * (kW4PanelRows / 2) <= (kWarps + 1) * 32)
    add_up(float2{});
  else
    add_up(float4{});
}

template <class T, int kNT>
cudaError_t logits_as(const W4MoeArgs &a, int splits, int n_counters, cudaStream_t s) {
  return launch_clusters(w4_moe_logits_kernel<T, kNT>, dim3(static_cast<unsigned>((a.E + 15) / 16 * splits)), kLogitWarps * 32, 0, splits, s, a, splits,
                         n_counters);
}

template <class T, int kGpb, bool kZeros>
cudaError_t experts_as(const W4MoeArgs &a, int sms, cudaStream_t s) {
  constexpr int kBytes = w4_block_bytes(kGpb, kZeros);
  // two CTAs to an SM of 228 KB, of which each CTA's static part and 1 KB of the system's go off
  constexpr int kStatic = 8192, kFit = (233472 / 2 - 1024 - kStatic) / (kWarps * kBytes), kDepth = kFit < kMaxDepth ? kFit : kMaxDepth;
  constexpr int kSmem = kDepth * kWarps * kBytes;
  static_assert(kDepth >= 2 && sizeof(PlanScratch) <= kSmem && kBytes >= 8 * kW4Pitch * 4, "rings, scratch and sums");
  static_assert(sizeof(Plan) + 2 * kWarps * kMaxDepth * 8 + kItems * 32 + kW4MoeMaxDim / kW4PanelRows * 2 + 256 <= kStatic, "static shared memory");
  const cudaError_t e = allow_smem<w4_moe_experts_kernel<T, kGpb, kZeros>>(kSmem);
  if (e != cudaSuccess) return e;
  // no more CTAs than panels
  const int64_t most = static_cast<int64_t>(a.T * a.topk + (a.sh13 ? (a.T + 7) / 8 : 0)) *
                       ((a.I + 31) / 32 + (a.H + kW4PanelRows - 1) / kW4PanelRows);
  const int64_t ctas = most < 2 * sms ? most : 2 * sms;
  return launch_pdl(w4_moe_experts_kernel<T, kGpb, kZeros>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), kSmem, s, a, kDepth);
}

template <class T>
cudaError_t moe_as(const W4MoeArgs &a, int group, bool zeros, int sms, cudaStream_t s) {
  const int tiles = (a.E + 15) / 16, chunks = (a.H + 31) / 32;
  int splits = sms / tiles;
  if (splits > chunks / kLogitWarps) splits = chunks / kLogitWarps;
  if (splits > kW4MaxRanks) splits = kW4MaxRanks;
  if (splits < 1) splits = 1;
  const int n = kW4MoeCounters + (a.H + kW4PanelRows - 1) / kW4PanelRows;
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
