// Host-side helpers shared by the translation units that implement the C ABI: error reporting,
// the per-device state and the TMA descriptors.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

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

struct DeviceInfo {
  bool ready = false;
  bool supported = false;
  int sms = 0;
  uint32_t *flags = nullptr;
};
nvfp4_status device_info(const char *fn, DeviceInfo **out);

// 2-D byte tensor (rows x row_bytes, row stride ld_bytes) read in boxes of
// 128 bytes x box_rows with the 128-byte swizzle.
nvfp4_status make_map(const char *fn, CUtensorMap *m, const void *base, int64_t row_bytes, int64_t rows,
                      int64_t ld_bytes, int box_rows, int box_bytes = 128,
                      CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B);

nvfp4_status check_ws(const char *fn, const void *ws, size_t ws_bytes, size_t need);

}  // namespace nvfp4
