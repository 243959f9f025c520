// Host-side helpers shared by the translation units that implement the C ABI: error reporting,
// the per-device state and the TMA descriptors.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>
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

// ---------------------------------------------------------------- checks of the operators around the experts

constexpr int64_t kMaxDim = int64_t(1) << 24;
constexpr int64_t kMaxArea = int64_t(1) << 40;

inline bool dtype16(int d) { return d == NVFP4_DT_BF16 || d == NVFP4_DT_FP16; }
inline bool dims_ok(int64_t a, int64_t b) { return a < kMaxDim && b < kMaxDim && a * b < kMaxArea; }

#define NV_DIMS(a, b)                                                                                \
  NV_REQUIRE(dims_ok(a, b), NVFP4_ERR_UNSUPPORTED_SHAPE, "sizes too large: %lld x %lld", (long long)(a), \
             (long long)(b))

// `rows` rows of `cols` elements of `bytes` bytes, `ld` elements apart, taken as the whole range from the first
// element to the last.
struct Span {
  const void *p;
  int64_t rows, ld, cols, bytes;
};
inline bool overlap(const Span &a, const Span &b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.cols <= 0 || b.cols <= 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  const uintptr_t a1 = a0 + static_cast<uintptr_t>(((a.rows - 1) * a.ld + a.cols) * a.bytes);
  const uintptr_t b1 = b0 + static_cast<uintptr_t>(((b.rows - 1) * b.ld + b.cols) * b.bytes);
  return a0 < b1 && b0 < a1;
}
inline Span flat(const void *p, int64_t n, int64_t bytes) { return {p, 1, n, n, bytes}; }

// Refuses what is written (outputs, the workspace) inside what is read, which other blocks may still be
// reading, and inside what else is written.
inline nvfp4_status check_disjoint(const char *fn, std::initializer_list<Span> written, std::initializer_list<Span> read) {
  for (auto w = written.begin(); w != written.end(); ++w) {
    for (const Span &r : read)
      if (overlap(*w, r)) return fail(NVFP4_ERR_INVALID_ARG, fn, "an output or the workspace overlaps an input");
    for (auto o = written.begin(); o != w; ++o)
      if (overlap(*w, *o)) return fail(NVFP4_ERR_INVALID_ARG, fn, "outputs and workspace overlap one another");
  }
  return NVFP4_OK;
}

}  // namespace nvfp4
