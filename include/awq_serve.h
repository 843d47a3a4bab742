/*
 * awq_serve.h -- C ABI of the serving operators next to the packed W4A16 product:
 *   - rows quantised to 8-bit integers (activations per token, weights per output channel),
 *     the product of two such matrices, and the linear layer that does both;
 *   - a paged key/value cache held in 4 bits by the same group quantiser as the weights, its
 *     write and read-back, and the attention that reads it.
 *
 * Conventions are those of awq_act.h: device pointers owned by the caller, caller-provided
 * workspaces, work enqueued on `stream` without synchronising, status codes, every check on
 * the host before any launch, calls thread-safe given distinct workspaces.  Launches are
 * kernels only, so a call may be captured into a HIP graph.
 */
#ifndef AWQ_SERVE_H
#define AWQ_SERVE_H

#include "awq_act.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of activations, outputs, biases, queries, keys and values. */
enum { AWQ_FP16 = 0, AWQ_BF16 = 1 };

/* ------------------------------------------------------------------------------------
 * Rows of 8-bit integers
 *   v[r][i] = A[r][i], A[r][i] / s[i] (AWQ_FOLD_DIVIDE: activations under the scales of a
 *             search [AWQ-notes §4.3]) or A[r][i] * s[i] (AWQ_FOLD_MULTIPLY: weights)
 *   step[r] = max_i |v[r][i]| / 127, a step of 0 replaced by 1
 *   code[r][i] = clamp(rint(v[r][i] / step[r]), -127, 127)  (the clamp acts on subnormal
 *             steps only)
 * in fp32, one rounding an operation, divisions correctly rounded, round half to even (the
 * symmetric quantiser of [AWQ-notes §2.3] with a group of one row).  A row that holds a NaN
 * or an infinity (also one that the fold makes) gets step NaN and codes 0, so that whatever
 * it is multiplied with is NaN.
 *   A          fp16 or bf16 [rows][cols], row stride lda >= cols elements; 2-byte aligned
 *              (16-byte loads are used where the base and lda allow them)
 *   s          fp32 [cols] or NULL
 *   codes_out  int8 [rows][ld_codes], 16-byte aligned, ld_codes a multiple of 16 and at
 *              least cols rounded up to 16; columns [cols, cols rounded up to 16) are
 *              written as zeros, later ones not at all
 *   steps_out  fp32 [rows]
 * rows, cols >= 0.
 * ---------------------------------------------------------------------------------- */
enum { AWQ_FOLD_DIVIDE = 0, AWQ_FOLD_MULTIPLY = 1 };
int awq_int8_quantize(const void* A, int64_t rows, int64_t cols, int64_t lda, int32_t dtype,
                      const float* s, int32_t fold, int8_t* codes_out, int64_t ld_codes,
                      float* steps_out, void* stream);

/* ------------------------------------------------------------------------------------
 * Product in 8-bit integers
 *   y[t][m] = float(sum_i xq[t][i] wq[m][i]) * xstep[t] * wstep[m] + bias[m]
 * The sum is exact (int32), then each operation, left to right, rounds once in fp32 and the
 * result once to the output type.
 *   xq     int8 [n_tokens][ldx], wq int8 [out][ldw], 16-byte aligned, strides multiples of 16
 *          and at least in_features rounded up to 16.  Columns from in_features up to that are
 *          read: they must be zero in xq or in wq (awq_int8_quantize writes zeros)
 *   xstep  fp32 [n_tokens], wstep fp32 [out], 4-byte aligned
 *   bias   [out] in the output's type, or NULL
 *   y      fp16 or bf16 [n_tokens][ldy], ldy >= out
 *   workspace  device, 256-byte aligned, awq_int8_matmul_workspace_bytes(...) bytes (0: may
 *          be NULL); contents unspecified before and after
 * in_features <= 131056 (the int32 sum cannot overflow), n_tokens, out_features < 2^31 with
 * n_tokens * ldx, out * ldw and n_tokens * ldy below 2^47; 0 tokens or outputs enqueue nothing,
 * in_features = 0 gives y = bias or 0.  Results do not depend on the launch configuration.
 * ---------------------------------------------------------------------------------- */
size_t awq_int8_matmul_workspace_bytes(int64_t n_tokens, int64_t out_features,
                                       int64_t in_features);
int awq_int8_matmul(const int8_t* xq, int64_t ldx, const float* xstep, int64_t n_tokens,
                    const int8_t* wq, int64_t ldw, const float* wstep, int64_t out_features,
                    int64_t in_features, const void* bias, int32_t dtype, void* y, int64_t ldy,
                    void* workspace, size_t workspace_bytes, void* stream);

/* The linear layer on floating activations: awq_int8_quantize of x (AWQ_FOLD_DIVIDE by s if
 * s is given) and awq_int8_matmul, with the same result bit for bit.  A few tokens run in one
 * launch that quantises the tokens on the fly; otherwise the codes go to the workspace.
 *   x fp16 or bf16 [n_tokens][ldx >= in_features], y, bias in the same type; other arguments
 *   as above. */
size_t awq_int8_linear_workspace_bytes(int64_t n_tokens, int64_t out_features,
                                       int64_t in_features);
int awq_int8_linear(const void* x, int64_t ldx, const float* s, int64_t n_tokens,
                    const int8_t* wq, int64_t ldw, const float* wstep, int64_t out_features,
                    int64_t in_features, const void* bias, int32_t dtype, void* y, int64_t ldy,
                    void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* AWQ_SERVE_H */
