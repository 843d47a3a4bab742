// C ABI of the MXFP4 operators, the norm and the read-back of 8-bit rows (awq_serve.h): argument checks,
// workspace carving, launches.  Every check that can fail runs on the host before anything is enqueued.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "awq_serve.h"
#include "mx_internal.h"
#include "serve_checks.h"
#include "serve_internal.h"

namespace {

constexpr int64_t kRows = awq::kMxMaxRows;

// Codes of `cols` columns in rows of ld bytes, with scale words in rows of lds.
bool codes_shape(int64_t rows, int64_t cols, int64_t ld, int64_t lds) {
  // a tile's panel of at most 256 rows is addressed with 32-bit offsets
  return rows >= 0 && rows <= kRows && cols >= 0 && cols <= awq::kMxMaxK &&
         ld >= awq::mx_code_bytes(cols) && ld % 16 == 0 && ld < (1 << 22) && lds >= rows &&
         lds % 4 == 0 && lds <= kRows && span_valid(rows, ld);
}

bool values_shape(int64_t rows, int64_t cols, int64_t ld) {
  return rows >= 0 && cols >= 0 && rows <= kMaxRows && cols <= kMaxRows && ld >= cols &&
         span_valid(rows, ld);
}

int matmul_shape(int64_t T, int64_t M, int64_t K, int64_t ldw, int64_t ldws, int64_t ldy) {
  if (T < 0 || T > kRows || !codes_shape(M, K, ldw, ldws) || ldy < M || !span_valid(T, ldy))
    return AWQ_E_SHAPE;
  return AWQ_OK;
}

bool matmul_sizes(int64_t T, int64_t M, int64_t K) {
  return T > 0 && M > 0 && K > 0 && T <= kRows && M <= kRows && K <= awq::kMxMaxK;
}

int norm_args(const void* x, int64_t ldx, const void* residual, int64_t ldr, int64_t rows, int64_t cols,
              int32_t dtype, const void* weight, int32_t weight_dtype, double eps, void* h_out,
              int64_t ldh, const void* y, awq::NormArgs* out) {
  if (!x || !y || (residual && !h_out)) return AWQ_E_NULL;
  if (!dtype_valid(dtype) || (weight && weight_dtype != AWQ_FP32 && weight_dtype != dtype) ||
      !(eps >= 1.1754943508222875e-38) || !isfinite(eps))
    return AWQ_E_CONFIG;
  if (!values_shape(rows, cols, ldx) || cols < 1 || rows > awq::kMaxBlocks ||
      (residual && (!values_shape(rows, cols, ldr) || !values_shape(rows, cols, ldh))))
    return AWQ_E_SHAPE;
  if (!aligned(x, 2) || !aligned(residual, 2) || (residual && !aligned(h_out, 2)) ||
      !aligned(weight, weight_dtype == AWQ_FP32 ? 4 : 2))
    return AWQ_E_ALIGN;
  awq::NormArgs a{};
  a.x = (const uint16_t*)x;
  a.ldx = ldx;
  a.r = (const uint16_t*)residual;
  a.ldr = ldr;
  a.h = residual ? (uint16_t*)h_out : nullptr;
  a.ldh = ldh;
  a.w = weight;
  a.w32 = weight_dtype == AWQ_FP32;
  a.bf16 = dtype == AWQ_BF16;
  a.eps = eps;
  a.inv_cols = 1.0 / (double)cols;
  a.rows = rows;
  a.cols = (int)cols;
  *out = a;
  return AWQ_OK;
}

int norm_launch(const awq::NormArgs& a, void* stream) {
  if (a.rows == 0) return AWQ_OK;
  if (int st = device_ptrs({a.x, a.r, a.h, a.w, a.y, a.scales})) return st;
  clear_pending_error();
  return hip_status(awq::launch_rmsnorm(a, (hipStream_t)stream));
}

}  // namespace

extern "C" {

int awq_int8_dequantize(const int8_t* codes, int64_t ld_codes, const float* steps, int64_t rows,
                        int64_t cols, int32_t dtype, void* out, int64_t ldo, void* stream) {
  if (!codes || !steps || !out) return AWQ_E_NULL;
  if (!dtype_valid(dtype)) return AWQ_E_CONFIG;
  if (!values_shape(rows, cols, ldo) || ld_codes < round16(cols) || ld_codes % 16 ||
      !span_valid(rows, ld_codes) || awq::values_blocks(rows, cols) > awq::kMaxBlocks)
    return AWQ_E_SHAPE;
  if (!aligned(codes, 16) || !aligned(steps, 4) || !aligned(out, 2)) return AWQ_E_ALIGN;
  if (rows == 0 || cols == 0) return AWQ_OK;
  if (int st = device_ptrs({codes, steps, out})) return st;
  clear_pending_error();
  return hip_status(awq::launch_int8_values(codes, ld_codes, steps, rows, (int)cols, dtype == AWQ_BF16,
                                            out, ldo, (hipStream_t)stream));
}

int awq_mxfp4_quantize(const void* A, int64_t rows, int64_t cols, int64_t lda, int32_t dtype,
                       const float* s, int32_t fold, uint8_t* codes_out, int64_t ld_codes,
                       uint8_t* scales_out, int64_t ld_scales, void* stream) {
  if (!A || !codes_out || !scales_out) return AWQ_E_NULL;
  if (!dtype_valid(dtype) || (fold != AWQ_FOLD_DIVIDE && fold != AWQ_FOLD_MULTIPLY))
    return AWQ_E_CONFIG;
  if (!values_shape(rows, cols, lda) || !codes_shape(rows, cols, ld_codes, ld_scales) ||
      awq::mxfp4_rows_blocks(rows, cols) > awq::kMaxBlocks)
    return AWQ_E_SHAPE;
  if (!aligned(A, 2) || !aligned(s, 4) || !aligned(codes_out, 16) || !aligned(scales_out, 16))
    return AWQ_E_ALIGN;
  if (rows == 0 || cols == 0) return AWQ_OK;
  if (int st = device_ptrs({A, s, codes_out, scales_out})) return st;
  clear_pending_error();
  return hip_status(awq::launch_mxfp4_rows(A, rows, (int)cols, lda, dtype == AWQ_BF16, s, fold, codes_out,
                                           ld_codes, (uint32_t*)scales_out, ld_scales,
                                           (hipStream_t)stream));
}

int awq_mxfp4_dequantize(const uint8_t* codes, int64_t ld_codes, const uint8_t* scales,
                         int64_t ld_scales, int64_t rows, int64_t cols, int32_t dtype, void* out,
                         int64_t ldo, void* stream) {
  if (!codes || !scales || !out) return AWQ_E_NULL;
  if (!dtype_valid(dtype)) return AWQ_E_CONFIG;
  if (!values_shape(rows, cols, ldo) || !codes_shape(rows, cols, ld_codes, ld_scales) ||
      awq::values_blocks(rows, cols) > awq::kMaxBlocks)
    return AWQ_E_SHAPE;
  if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(out, 2)) return AWQ_E_ALIGN;
  if (rows == 0 || cols == 0) return AWQ_OK;
  if (int st = device_ptrs({codes, scales, out})) return st;
  clear_pending_error();
  return hip_status(awq::launch_mxfp4_values(codes, ld_codes, (const uint32_t*)scales, ld_scales, rows,
                                             (int)cols, dtype == AWQ_BF16, out, ldo,
                                             (hipStream_t)stream));
}

int awq_mxfp4_matmul(const uint8_t* xc, int64_t ldx, const uint8_t* xs, int64_t ldxs, int64_t n_tokens,
                     const uint8_t* wc, int64_t ldw, const uint8_t* ws, int64_t ldws,
                     int64_t out_features, int64_t in_features, const void* bias, int32_t dtype, void* y,
                     int64_t ldy, void* stream) {
  const int64_t T = n_tokens, M = out_features, K = in_features;
  if (!xc || !xs || !wc || !ws || !y) return AWQ_E_NULL;
  if (!dtype_valid(dtype)) return AWQ_E_CONFIG;
  int st = matmul_shape(T, M, K, ldw, ldws, ldy);
  if (st) return st;
  if (!codes_shape(T, K, ldx, ldxs)) return AWQ_E_SHAPE;
  if (!aligned(xc, 16) || !aligned(wc, 16) || !aligned(xs, 16) || !aligned(ws, 16) ||
      !aligned(bias, 2) || !aligned(y, 2))
    return AWQ_E_ALIGN;
  if (T == 0 || M == 0) return AWQ_OK;
  if ((st = device_ptrs({xc, xs, wc, ws, bias, y}))) return st;
  clear_pending_error();
  const awq::MxArgs a{xc, ldx, (const uint32_t*)xs, ldxs, wc, ldw, (const uint32_t*)ws, ldws, bias, y, ldy,
                      (int)T, (int)M, (int)awq::mx_code_bytes(K), dtype == AWQ_BF16};
  return hip_status(awq::launch_mxfp4_matmul(a, (hipStream_t)stream));
}

size_t awq_mxfp4_linear_workspace_bytes(int64_t T, int64_t M, int64_t K) {
  if (!matmul_sizes(T, M, K) || awq::mxfp4_linear_fused(T, M, K)) return 0;
  return round_up((size_t)T * (size_t)awq::mx_code_bytes(K), kAlign) +
         round_up((size_t)awq::mx_words(K) * (size_t)((T + 3) / 4 * 4) * 4, kAlign);
}

int awq_mxfp4_linear(const void* x, int64_t ldx, const float* s, int64_t n_tokens, const uint8_t* wc,
                     int64_t ldw, const uint8_t* ws, int64_t ldws, int64_t out_features,
                     int64_t in_features, const void* bias, int32_t dtype, void* y, int64_t ldy,
                     void* workspace, size_t workspace_bytes, void* stream) {
  const int64_t T = n_tokens, M = out_features, K = in_features;
  if (!x || !wc || !ws || !y) return AWQ_E_NULL;
  if (!dtype_valid(dtype)) return AWQ_E_CONFIG;
  int st = matmul_shape(T, M, K, ldw, ldws, ldy);
  if (st) return st;
  if (!values_shape(T, K, ldx) || awq::mxfp4_rows_blocks(T, K) > awq::kMaxBlocks) return AWQ_E_SHAPE;
  const size_t need = awq_mxfp4_linear_workspace_bytes(T, M, K);
  if (need && (!workspace || workspace_bytes < need)) return AWQ_E_WORKSPACE;
  if (!aligned(x, 2) || !aligned(s, 4) || !aligned(wc, 16) || !aligned(ws, 16) || !aligned(bias, 2) ||
      !aligned(y, 2) || (need && !aligned(workspace, kAlign)))
    return AWQ_E_ALIGN;
  if (T == 0 || M == 0) return AWQ_OK;
  if ((st = device_ptrs({x, s, wc, ws, bias, y, need ? workspace : nullptr}))) return st;
  clear_pending_error();
  const bool bf16 = dtype == AWQ_BF16;
  const int64_t KB = awq::mx_code_bytes(K), lds = (T + 3) / 4 * 4;
  awq::MxArgs a{nullptr, KB, nullptr, lds, wc, ldw, (const uint32_t*)ws, ldws, bias, y, ldy,
                (int)T, (int)M, (int)KB, bf16};
  if (K > 0 && awq::mxfp4_linear_fused(T, M, K))
    return hip_status(awq::launch_mxfp4_linear_fused(a, x, ldx, s, (int)K, (hipStream_t)stream));
  uint8_t* p = (uint8_t*)workspace;
  const size_t n_codes = round_up((size_t)T * (size_t)KB, kAlign);
  a.x = p;
  a.xs = (const uint32_t*)(p + n_codes);
  hipError_t e = awq::launch_mxfp4_rows(x, T, (int)K, ldx, bf16, s, awq::kFoldDivide, p, KB,
                                        (uint32_t*)(p + n_codes), lds, (hipStream_t)stream);
  if (e != hipSuccess) return hip_status(e);
  return hip_status(awq::launch_mxfp4_matmul(a, (hipStream_t)stream));
}

int awq_rmsnorm(const void* x, int64_t ldx, const void* residual, int64_t ldr, int64_t rows,
                int64_t cols, int32_t dtype, const void* weight, int32_t weight_dtype, double eps,
                void* h_out, int64_t ldh, void* y, int64_t ldy, void* stream) {
  awq::NormArgs a;
  if (int st = norm_args(x, ldx, residual, ldr, rows, cols, dtype, weight, weight_dtype, eps, h_out, ldh,
                         y, &a))
    return st;
  if (!values_shape(rows, cols, ldy)) return AWQ_E_SHAPE;
  if (!aligned(y, 2)) return AWQ_E_ALIGN;
  a.out = awq::kNormSame;
  a.y = y;
  a.ldy = ldy;
  return norm_launch(a, stream);
}

int awq_rmsnorm_int8(const void* x, int64_t ldx, const void* residual, int64_t ldr, int64_t rows,
                     int64_t cols, int32_t dtype, const void* weight, int32_t weight_dtype, double eps,
                     void* h_out, int64_t ldh, int8_t* codes_out, int64_t ld_codes, float* steps_out,
                     void* stream) {
  awq::NormArgs a;
  if (int st = norm_args(x, ldx, residual, ldr, rows, cols, dtype, weight, weight_dtype, eps, h_out, ldh,
                         codes_out, &a))
    return st;
  if (!steps_out) return AWQ_E_NULL;
  if (ld_codes < round16(cols) || ld_codes % 16 || !span_valid(rows, ld_codes)) return AWQ_E_SHAPE;
  if (!aligned(codes_out, 16) || !aligned(steps_out, 4)) return AWQ_E_ALIGN;
  a.out = awq::kNormInt8;
  a.y = codes_out;
  a.ldy = ld_codes;
  a.scales = steps_out;
  return norm_launch(a, stream);
}

int awq_rmsnorm_mxfp4(const void* x, int64_t ldx, const void* residual, int64_t ldr, int64_t rows,
                      int64_t cols, int32_t dtype, const void* weight, int32_t weight_dtype, double eps,
                      void* h_out, int64_t ldh, uint8_t* codes_out, int64_t ld_codes,
                      uint8_t* scales_out, int64_t ld_scales, void* stream) {
  awq::NormArgs a;
  if (int st = norm_args(x, ldx, residual, ldr, rows, cols, dtype, weight, weight_dtype, eps, h_out, ldh,
                         codes_out, &a))
    return st;
  if (!scales_out) return AWQ_E_NULL;
  if (!codes_shape(rows, cols, ld_codes, ld_scales)) return AWQ_E_SHAPE;
  if (!aligned(codes_out, 16) || !aligned(scales_out, 16)) return AWQ_E_ALIGN;
  a.out = awq::kNormMxfp4;
  a.y = codes_out;
  a.ldy = ld_codes;
  a.scales = scales_out;
  a.ld_scales = ld_scales;
  return norm_launch(a, stream);
}

}  // extern "C"
