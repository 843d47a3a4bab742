// C ABI of the serving operators (awq_serve.h): argument checks, workspace carving, launches.
// Every check that can fail runs on the host before anything is enqueued.
#include <hip/hip_runtime.h>

#include <stdint.h>
#include <string.h>

#include "awq_serve.h"
#include "serve_internal.h"

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
int device_ptrs(std::initializer_list<const void*> ps) {
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

int int8_shape(int64_t T, int64_t M, int64_t K, int64_t ldw, int64_t ldy) {
  if (T < 0 || M < 0 || K < 0 || T > kMaxRows || M > kMaxRows || K > awq::kInt8MaxK)
    return AWQ_E_SHAPE;
  // a tile's panel of at most 256 rows is addressed with 32-bit offsets
  if (ldw < round16(K) || ldw % 16 || ldw >= (1 << 22) || ldy < M) return AWQ_E_SHAPE;
  if (!span_valid(M, ldw) || !span_valid(T, ldy)) return AWQ_E_SHAPE;
  return AWQ_OK;
}

}  // namespace

extern "C" {

int awq_int8_quantize(const void* A, int64_t rows, int64_t cols, int64_t lda, int32_t dtype,
                      const float* s, int32_t fold, int8_t* codes_out, int64_t ld_codes,
                      float* steps_out, void* stream) {
  if (!A || !codes_out || !steps_out) return AWQ_E_NULL;
  if (!dtype_valid(dtype) || (fold != AWQ_FOLD_DIVIDE && fold != AWQ_FOLD_MULTIPLY))
    return AWQ_E_CONFIG;
  if (rows < 0 || cols < 0 || rows > kMaxRows || cols > kMaxRows || lda < cols ||
      ld_codes < round16(cols) || ld_codes % 16 || !span_valid(rows, lda) ||
      !span_valid(rows, ld_codes))
    return AWQ_E_SHAPE;
  if (!aligned(A, 2) || !aligned(s, 4) || !aligned(codes_out, 16) || !aligned(steps_out, 4))
    return AWQ_E_ALIGN;
  if (rows == 0) return AWQ_OK;
  if (int st = device_ptrs({A, s, codes_out, steps_out})) return st;
  clear_pending_error();
  return hip_status(awq::launch_int8_rows(A, rows, (int)cols, lda, dtype == AWQ_BF16, s, fold,
                                          codes_out, ld_codes, steps_out, (hipStream_t)stream));
}

size_t awq_int8_matmul_workspace_bytes(int64_t T, int64_t M, int64_t K) {
  if (T <= 0 || M <= 0 || K <= 0 || T > kMaxRows || M > kMaxRows || K > awq::kInt8MaxK) return 0;
  return round_up(awq::int8_matmul_workspace(T, M, K), kAlign);
}

int awq_int8_matmul(const int8_t* xq, int64_t ldx, const float* xstep, int64_t n_tokens,
                    const int8_t* wq, int64_t ldw, const float* wstep, int64_t out_features,
                    int64_t in_features, const void* bias, int32_t dtype, void* y, int64_t ldy,
                    void* workspace, size_t workspace_bytes, void* stream) {
  const int64_t T = n_tokens, M = out_features, K = in_features;
  if (!xq || !xstep || !wq || !wstep || !y) return AWQ_E_NULL;
  if (!dtype_valid(dtype)) return AWQ_E_CONFIG;
  int st = int8_shape(T, M, K, ldw, ldy);
  if (st) return st;
  if (ldx < round16(K) || ldx % 16 || ldx >= (1 << 22) || !span_valid(T, ldx)) return AWQ_E_SHAPE;
  const size_t need = awq_int8_matmul_workspace_bytes(T, M, K);
  if (need && (!workspace || workspace_bytes < need)) return AWQ_E_WORKSPACE;
  if (!aligned(xq, 16) || !aligned(wq, 16) || !aligned(xstep, 4) || !aligned(wstep, 4) ||
      !aligned(bias, 2) || !aligned(y, 2) || (need && !aligned(workspace, kAlign)))
    return AWQ_E_ALIGN;
  if (T == 0 || M == 0) return AWQ_OK;
  if ((st = device_ptrs({xq, xstep, wq, wstep, bias, y, need ? workspace : nullptr}))) return st;
  clear_pending_error();
  const awq::Int8Args a{xq, ldx, xstep, wq, ldw, wstep, bias, y, ldy,
                        (int)T, (int)M, (int)round16(K), dtype == AWQ_BF16};
  return hip_status(awq::launch_int8_matmul(a, workspace, (hipStream_t)stream));
}

size_t awq_int8_linear_workspace_bytes(int64_t T, int64_t M, int64_t K) {
  if (T <= 0 || M <= 0 || K < 0 || T > kMaxRows || M > kMaxRows || K > awq::kInt8MaxK) return 0;
  return round_up((size_t)T * (size_t)round16(K), kAlign) + round_up((size_t)T * 4, kAlign) +
         awq_int8_matmul_workspace_bytes(T, M, K);
}

int awq_int8_linear(const void* x, int64_t ldx, const float* s, int64_t n_tokens,
                    const int8_t* wq, int64_t ldw, const float* wstep, int64_t out_features,
                    int64_t in_features, const void* bias, int32_t dtype, void* y, int64_t ldy,
                    void* workspace, size_t workspace_bytes, void* stream) {
  const int64_t T = n_tokens, M = out_features, K = in_features;
  if (!x || !wq || !wstep || !y) return AWQ_E_NULL;
  if (!dtype_valid(dtype)) return AWQ_E_CONFIG;
  int st = int8_shape(T, M, K, ldw, ldy);
  if (st) return st;
  if (ldx < K || !span_valid(T, ldx)) return AWQ_E_SHAPE;
  const size_t need = awq_int8_linear_workspace_bytes(T, M, K);
  if (need && (!workspace || workspace_bytes < need)) return AWQ_E_WORKSPACE;
  if (!aligned(x, 2) || !aligned(s, 4) || !aligned(wq, 16) || !aligned(wstep, 4) ||
      !aligned(bias, 2) || !aligned(y, 2) || (need && !aligned(workspace, kAlign)))
    return AWQ_E_ALIGN;
  if (T == 0 || M == 0) return AWQ_OK;
  if ((st = device_ptrs({x, s, wq, wstep, bias, y, need ? workspace : nullptr}))) return st;
  clear_pending_error();
  char* ws = (char*)workspace;
  int8_t* xq = (int8_t*)ws;
  ws += round_up((size_t)T * (size_t)round16(K), kAlign);
  float* xstep = (float*)ws;
  ws += round_up((size_t)T * 4, kAlign);
  if ((st = hip_status(awq::launch_int8_rows(x, T, (int)K, ldx, dtype == AWQ_BF16, s,
                                             AWQ_FOLD_DIVIDE, xq, round16(K), xstep,
                                             (hipStream_t)stream))))
    return st;
  const awq::Int8Args a{xq, round16(K), xstep, wq, ldw, wstep, bias, y, ldy,
                        (int)T, (int)M, (int)round16(K), dtype == AWQ_BF16};
  return hip_status(awq::launch_int8_matmul(a, ws, (hipStream_t)stream));
}

}  // extern "C"
