// Host-side helpers shared by the translation units that implement the C ABI: error reporting,
// the per-device state and the TMA descriptors.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <mutex>

#include "internal.h"

namespace nvfp4 {

nvfp4_status fail(nvfp4_status st, const char *fn, const char *fmt, ...);
nvfp4_status cuda_fail(const char *fn, cudaError_t e, const char *what);

#define NV_REQUIRE(cond, status, ...) \
  do {                                \
    if (!(cond)) return fail(status, __func__, __VA_ARGS__); \
  } while (0)

#define NV_CUDA(expr, what)                          \
  do {                                               \
    cudaError_t e_ = (expr);                         \
    if (e_ != cudaSuccess) return cuda_fail(__func__, e_, what); \
  } while (0)

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }
inline int64_t round_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

// A CTA-pair launch: its stream, the capture it is part of (0 outside one; ids), and an event behind it.
struct PairLaunch {
  cudaEvent_t event = nullptr;
  unsigned long long stream = 0, capture = 0;
  bool made = false;
};

// Stream captures that may go on at once on a device with their branches' pair launches in order.
constexpr int kMaxPairCaptures = 16;

struct DeviceInfo {
  bool ready = false;
  bool supported = false;
  int sms = 0;
  uint32_t *flags = nullptr;
  std::mutex pair_mutex;
  PairLaunch pair_last;                       // the last one outside captures
  PairLaunch pair_captured[kMaxPairCaptures];  // and of each of the latest captures
};
nvfp4_status device_info(const char *fn, DeviceInfo **out);

// Launches of kernels on CTA pairs (tcgen05 cta_group::2) run one after the other on a device, whatever
// streams they are queued on: two that overlap, one taking over the SMs and tensor memory that the
// other leaves pair by pair, once stopped making progress (tile_gemm.cuh).  A launch on another stream
// than the last one's waits for an event behind that one; inside a stream capture the same holds
// between the branches of the captured graph.  Launches of different graphs, and of a graph and a stream,
// are not ordered by this: the caller replays them in turn.
cudaError_t pair_turn_begin(DeviceInfo *d, cudaStream_t s, PairLaunch *now, PairLaunch **last);
cudaError_t pair_turn_end(cudaStream_t s, const PairLaunch &now, PairLaunch *last);
template <class Launch>
cudaError_t in_pair_turn(DeviceInfo *d, cudaStream_t s, Launch launch) {
  std::lock_guard<std::mutex> lock(d->pair_mutex);  // over the launch: the host's order is the device's
  PairLaunch now, *last;
  cudaError_t e = pair_turn_begin(d, s, &now, &last);
  if (e == cudaSuccess) e = launch();
  return e == cudaSuccess ? pair_turn_end(s, now, last) : e;
}

// 2-D byte tensor (rows x row_bytes, row stride ld_bytes) read in boxes of
// 128 bytes x box_rows with the 128-byte swizzle.
nvfp4_status make_map(const char *fn, CUtensorMap *m, const void *base, int64_t row_bytes, int64_t rows,
                      int64_t ld_bytes, int box_rows, int box_bytes = 128,
                      CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B);

nvfp4_status check_ws(const char *fn, const void *ws, size_t ws_bytes, size_t need);

}  // namespace nvfp4
