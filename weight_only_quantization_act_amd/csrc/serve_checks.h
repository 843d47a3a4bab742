// Argument checks shared by the C ABI of the serving operators (host code).
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>
#include <string.h>

#include <initializer_list>

#include "awq_serve.h"

namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 512;  // rounded-up row counts stay in 32 bits
constexpr int64_t kMaxSpan = (int64_t)1 << 47;          // elements from the first to the last row

inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline int64_t round16(int64_t k) { return (k + 15) / 16 * 16; }
inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline int hip_status(hipError_t e) { return e == hipSuccess ? AWQ_OK : AWQ_E_HIP; }
inline void clear_pending_error() { (void)hipGetLastError(); }
inline bool dtype_valid(int32_t d) { return d == AWQ_FP16 || d == AWQ_BF16; }
inline bool span_valid(int64_t rows, int64_t ld) { return rows == 0 || ld <= kMaxSpan / rows; }

// The pointers that a launch dereferences must be device (or managed) memory; NULLs are
// optional arguments.
inline int device_ptrs(std::initializer_list<const void*> ps) {
  for (const void* p : ps) {
    if (!p) continue;
    hipPointerAttribute_t attr;
    memset(&attr, 0, sizeof(attr));
    if (hipPointerGetAttributes(&attr, p) != hipSuccess) {
      (void)hipGetLastError();
      return AWQ_E_DEVICE;
    }
    if (attr.type != hipMemoryTypeDevice && attr.type != hipMemoryTypeManaged) return AWQ_E_DEVICE;
  }
  return AWQ_OK;
}

}  // namespace
