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
 *   xq     int8 [n_tokens][ldx], wq int8 [out][ldw], 16-byte aligned, strides multiples of 16,
 *          at least in_features rounded up to 16 and below 2^22.  Columns from in_features up to that are
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
 * s is given) and awq_int8_matmul, with the same result bit for bit.  One token of up to
 * 16384 columns runs in one launch that quantises it on the fly; otherwise the codes go to the
 * workspace.
 *   x fp16 or bf16 [n_tokens][ldx >= in_features], y, bias in the same type; other arguments
 *   as above. */
size_t awq_int8_linear_workspace_bytes(int64_t n_tokens, int64_t out_features,
                                       int64_t in_features);
int awq_int8_linear(const void* x, int64_t ldx, const float* s, int64_t n_tokens,
                    const int8_t* wq, int64_t ldw, const float* wstep, int64_t out_features,
                    int64_t in_features, const void* bias, int32_t dtype, void* y, int64_t ldy,
                    void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------------------
 * Key/value cache in 4 bits
 *   Keys and values of a token and head are quantised along head_dim in groups of group_size
 *   channels by the quantiser of awq_quantize_pack with w_bit 4 and no channel scales (fp32,
 *   one rounding an operation; symmetric or zero-point); a value reads as
 *   (code - zero) * fp16(step) [AWQ-blog §1.2, §2.1; AutoAWQ-70B §四 (metadata per group)].
 *   A group whose range is not finite (it holds a NaN or an infinity, or the range overflows) is
 *   stored with step NaN, codes and zero 0.
 *   A finite step beyond fp16's 65504 (bf16 ranges of a million) is stored as infinity: such values
 *   read as infinite or NaN, and a key of such a step makes the rows that see it NaN.
 *
 *   cache        uint8 [n_pages][kv_heads][record], 16-byte aligned; record =
 *                awq_kv4_record_bytes(cfg).  With D = head_dim, P = page_size, g = group_size,
 *                G = D / g a record is
 *                  K codes   P rows of D / 2 bytes: [q 0..3][j < G][u < g / 32] 32-bit words;
 *                            nibble n (bits 4 n) is channel j g + q g / 4 + 8 u + n
 *                  V codes   P / 8 blocks of 8 tokens: [h < D / 64][r < 16][i < 4] 32-bit words;
 *                            the low half is token 2 i of the block, the high half 2 i + 1,
 *                            nibble c of a half is channel 16 (4 h + c) + r
 *                  K params  [G][P] pairs of fp16 step, fp16 zero
 *                  V params  the same
 *   block_table  int32 [n_seqs][max_blocks] (row-major): token t of sequence b is token
 *                t mod P of page block_table[b][t / P].  Entries past a sequence's length are
 *                not read.  Entries outside [0, n_pages) and positions past max_blocks are
 *                no memory: a write there is dropped, and keys there are masked
 *   seq_lens     int32 [n_seqs]: tokens of each sequence, the new ones included
 *   q_start      int32 [n_seqs + 1], ascending from 0: rows q_start[b] .. q_start[b + 1] - 1 of
 *                k, v and q are the last tokens of sequence b (positions seq_lens[b] - count
 *                .. seq_lens[b] - 1).  Rows at negative positions do not exist: they are not
 *                written, read as zeros and attend to nothing.  Nor do rows past n_tokens
 *   k, v, q      fp16 or bf16 [token][head][head_dim], unit stride in head_dim, token and head
 *                strides in elements (multiples of 8, 0 .. 2^31, 16-byte aligned base)
 * n_seqs <= 65535, n_pages < 2^31, max_blocks x page_size < 2^31.  A call that would take 2^31
 * blocks or so (n_tokens x kv_heads x head_dim 2^42, n_seqs x kv_heads 2^30) is AWQ_E_SHAPE.
 * All sizes are device data except the bounds named below; a call may be captured and replayed
 * while lengths and tables change within those bounds.
 * ---------------------------------------------------------------------------------- */
typedef struct awq_kv4_config {
  int32_t head_dim;   /* 64 or 128                             */
  int32_t kv_heads;   /* 1 .. 65535                            */
  int32_t page_size;  /* tokens a page: 16, 32, 64, 128 or 256 */
  int32_t group_size; /* 32, 64 or 128, at most head_dim       */
  int32_t zero_point; /* 0 = symmetric, 1 = zero-point         */
} awq_kv4_config;

/* Bytes of one page of one head, or 0 for an invalid configuration. */
size_t awq_kv4_record_bytes(const awq_kv4_config* cfg);

/* Quantise the new tokens' keys and values (n_tokens rows of k and v, rows past
 * q_start[n_seqs] ignored) into the cache. */
int awq_kv4_append(const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                   int64_t v_token_stride, int64_t v_head_stride, int64_t n_tokens, int32_t dtype,
                   void* cache, int64_t n_pages, const int32_t* block_table, int64_t n_seqs,
                   int64_t max_blocks, const int32_t* seq_lens, const int32_t* q_start,
                   const awq_kv4_config* cfg, void* stream);

/* The stored values of the same rows: k_out and v_out [n_tokens][kv_heads][head_dim], contiguous,
 * 16-byte aligned, (code - zero) * step in fp32 rounded once to dtype; rows that do not exist
 * are zeros. */
int awq_kv4_read(const void* cache, int64_t n_pages, const int32_t* block_table, int64_t n_seqs,
                 int64_t max_blocks, const int32_t* seq_lens, const int32_t* q_start,
                 int64_t n_tokens, const awq_kv4_config* cfg, int32_t dtype, void* k_out,
                 void* v_out, void* stream);

/* Attention of the rows of q over the cached keys and values:
 *   out[r][h] = sum_t p_t v_t,  p = softmax over t of scale q[r][h] . k_t,
 *   t <= position of r (and t > position - window if window > 0), with key/value head
 *   h / (heads / kv_heads); lse[r][h] = log sum_t exp(scale q . k_t).
 * A row without keys gives out 0 and lse -infinity.  Scores, softmax statistics and sums are
 * fp32; q enters the products in fp16, each row scaled by a power of two (exact but for parts
 * 2^-24 and more below the row's largest), the probabilities times the value's step rounded to
 * fp16 with 2^-11 relative error (or 2^-36 of the largest finite value step that the row sees);
 * keys and values enter as the integers code - zero, with zeros 0 .. 15; where max_q x heads /
 * kv_heads is at most 16, as 16 + code and 16 + zero, whose fp32 sums round at sum p step (code +
 * zero + 32) and are subtracted at the end.  A NaN or infinity in a row of q or a NaN in a key
 * that it sees makes the row NaN, one in a value the channels of its group; keys that a row does
 * not see cost it no precision either.  The order of every sum is fixed: results repeat bit for
 * bit for the same bounds.
 *   q        as above, n_tokens rows, heads a multiple of kv_heads
 *   max_q    bound on the rows of one sequence, max_len bound on seq_lens (both host values, up to
 *            2^30: they size the launch; rows and keys beyond them are not computed)
 *   scale    finite, > 0; window 0 or more
 *   out      [n_tokens][heads][head_dim] contiguous, q's type, 16-byte aligned; rows past
 *            q_start[n_seqs] are not written
 *   lse_out  fp32 [n_tokens][heads] or NULL
 *   workspace  device, 256-byte aligned, awq_kv4_attention_workspace_bytes(...) bytes (0: may
 *            be NULL), contents unspecified before and after */
size_t awq_kv4_attention_workspace_bytes(int64_t n_tokens, int64_t n_seqs, int64_t heads,
                                         const awq_kv4_config* cfg, int64_t max_q,
                                         int64_t max_len);
int awq_kv4_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                      int64_t n_tokens, int64_t heads, int32_t dtype, const void* cache,
                      int64_t n_pages, const int32_t* block_table, int64_t n_seqs,
                      int64_t max_blocks, const int32_t* seq_lens, const int32_t* q_start,
                      const awq_kv4_config* cfg, int64_t max_q, int64_t max_len, float scale,
                      int64_t window, void* out, float* lse_out, void* workspace,
                      size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* AWQ_SERVE_H */
