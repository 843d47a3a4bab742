// C ABI of the serving operators (awq_serve.h): argument checks, workspace carving, launches.
// Every check that can fail runs on the host before anything is enqueued.
#include <hip/hip_runtime.h>

#include <stdint.h>
#include <string.h>

#include <initializer_list>

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

bool kv4_valid(const awq_kv4_config* c) {
  if (!c) return false;
  if (c->head_dim != 64 && c->head_dim != 128) return false;
  if (c->kv_heads < 1 || c->kv_heads > 65535) return false;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return false;
  if (c->group_size != 32 && c->group_size != 64 && c->group_size != 128) return false;
  if (c->group_size > c->head_dim) return false;
  return c->zero_point == 0 || c->zero_point == 1;
}

// Sizes common to the cache's calls; fills the launch description.
int kv4_cache(const void* cache, int64_t n_pages, const int32_t* table, int64_t n_seqs,
              int64_t max_blocks, const int32_t* lens, const int32_t* starts, int64_t n_tokens,
              const awq_kv4_config* cfg, awq::Kv4Cache* out) {
  if (!cache || !table || !lens || !starts || !cfg) return AWQ_E_NULL;
  if (!kv4_valid(cfg)) return AWQ_E_CONFIG;
  // n_seqs is a grid dimension; positions are 32-bit
  if (n_pages < 1 || n_pages > 0x7fffffff || n_seqs < 0 || n_seqs > 65535 || max_blocks < 1 ||
      max_blocks > 0x7fffffff / cfg->page_size || n_tokens < 0 || n_tokens > kMaxRows)
    return AWQ_E_SHAPE;
  if (!aligned(cache, 16) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(starts, 4))
    return AWQ_E_ALIGN;
  int log2p = 0;
  while ((1 << log2p) < cfg->page_size) ++log2p;
  *out = awq::Kv4Cache{(uint8_t*)cache, n_pages, table, lens, starts, (int)n_seqs, (int)max_blocks,
                       cfg->kv_heads, cfg->head_dim, cfg->group_size, log2p, cfg->zero_point,
                       awq::kv4_record(cfg->head_dim, cfg->group_size, cfg->page_size)};
  return AWQ_OK;
}

// Rows of heads: 16-byte pieces from any (token, head); spans stay far from 64-bit overflow.
int kv4_rows(const void* p, int64_t token_stride, int64_t head_stride) {
  if (token_stride < 0 || head_stride < 0 || token_stride % 8 || head_stride % 8 ||
      token_stride > ((int64_t)1 << 31) || head_stride > ((int64_t)1 << 31))
    return AWQ_E_SHAPE;
  return aligned(p, 16) ? AWQ_OK : AWQ_E_ALIGN;
}

int attention_shape(int64_t n_tokens, int64_t n_seqs, int64_t heads, const awq_kv4_config* cfg,
                    int64_t max_q, int64_t max_len) {
  if (n_tokens < 0 || n_tokens > kMaxRows || n_seqs < 0 || n_seqs > 65535 || max_q < 0 ||
      max_len < 0 || max_len > ((int64_t)1 << 30) || max_q > ((int64_t)1 << 30))
    return AWQ_E_SHAPE;
  if (heads < 1 || heads > 65535 || heads % cfg->kv_heads) return AWQ_E_SHAPE;
  // columns of a key head and (token, head) rows are counted in 32 bits
  if (max_q * (heads / cfg->kv_heads) > ((int64_t)1 << 30)) return AWQ_E_SHAPE;
  if (n_tokens > (((int64_t)1 << 31) - 1024) / heads) return AWQ_E_SHAPE;
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
  // planned, as the launch is, from the columns that are read: rows of whole 16-byte chunks
  return round_up(awq::int8_matmul_workspace(T, M, round16(K)), kAlign);
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
  if (awq::int8_linear_fused(T, round16(K))) return 0;
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
  if (awq::int8_linear_fused(T, round16(K))) {
    const awq::Int8Args a{nullptr, 0, nullptr, wq, ldw, wstep, bias, y, ldy,
                          (int)T, (int)M, (int)round16(K), dtype == AWQ_BF16};
    return hip_status(awq::launch_int8_linear_fused(a, x, s, (int)K, (hipStream_t)stream));
  }
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

size_t awq_kv4_record_bytes(const awq_kv4_config* cfg) {
  return kv4_valid(cfg) ? awq::kv4_record(cfg->head_dim, cfg->group_size, cfg->page_size) : 0;
}

int awq_kv4_append(const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                   int64_t v_token_stride, int64_t v_head_stride, int64_t n_tokens, int32_t dtype,
                   void* cache, int64_t n_pages, const int32_t* block_table, int64_t n_seqs,
                   int64_t max_blocks, const int32_t* seq_lens, const int32_t* q_start,
                   const awq_kv4_config* cfg, void* stream) {
  if (!k || !v) return AWQ_E_NULL;
  awq::Kv4Cache c;
  int st = kv4_cache(cache, n_pages, block_table, n_seqs, max_blocks, seq_lens, q_start, n_tokens,
                     cfg, &c);
  if (st) return st;
  if (!dtype_valid(dtype)) return AWQ_E_CONFIG;
  if ((st = kv4_rows(k, k_token_stride, k_head_stride)) ||
      (st = kv4_rows(v, v_token_stride, v_head_stride)))
    return st;
  if (n_tokens == 0 || n_seqs == 0) return AWQ_OK;
  if (awq::kv4_store_blocks(n_tokens, cfg->head_dim, (int)n_seqs, cfg->kv_heads) > awq::kMaxBlocks)
    return AWQ_E_SHAPE;
  if ((st = device_ptrs({k, v, cache, block_table, seq_lens, q_start}))) return st;
  clear_pending_error();
  return hip_status(awq::launch_kv4_append(c, k, k_token_stride, k_head_stride, v, v_token_stride,
                                           v_head_stride, n_tokens, dtype == AWQ_BF16,
                                           (hipStream_t)stream));
}

int awq_kv4_read(const void* cache, int64_t n_pages, const int32_t* block_table, int64_t n_seqs,
                 int64_t max_blocks, const int32_t* seq_lens, const int32_t* q_start,
                 int64_t n_tokens, const awq_kv4_config* cfg, int32_t dtype, void* k_out,
                 void* v_out, void* stream) {
  if (!k_out || !v_out) return AWQ_E_NULL;
  awq::Kv4Cache c;
  int st = kv4_cache(cache, n_pages, block_table, n_seqs, max_blocks, seq_lens, q_start, n_tokens,
                     cfg, &c);
  if (st) return st;
  if (!dtype_valid(dtype)) return AWQ_E_CONFIG;
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return AWQ_E_ALIGN;
  if (n_tokens == 0) return AWQ_OK;
  if (awq::kv4_store_blocks(n_tokens, cfg->head_dim, (int)n_seqs, cfg->kv_heads) > awq::kMaxBlocks)
    return AWQ_E_SHAPE;
  if ((st = device_ptrs({cache, block_table, seq_lens, q_start, k_out, v_out}))) return st;
  clear_pending_error();
  return hip_status(awq::launch_kv4_read(c, n_tokens, dtype == AWQ_BF16, k_out, v_out,
                                         (hipStream_t)stream));
}

size_t awq_kv4_attention_workspace_bytes(int64_t n_tokens, int64_t n_seqs, int64_t heads,
                                         const awq_kv4_config* cfg, int64_t max_q,
                                         int64_t max_len) {
  if (!kv4_valid(cfg) || attention_shape(n_tokens, n_seqs, heads, cfg, max_q, max_len)) return 0;
  if (n_tokens == 0 || n_seqs == 0 || max_q == 0) return 0;
  return round_up(awq::kv4_workspace_any_window(n_tokens, n_seqs, (int)heads, cfg->kv_heads, cfg->head_dim,
                                                cfg->group_size, max_q, max_len),
                  kAlign);
}

int awq_kv4_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                      int64_t n_tokens, int64_t heads, int32_t dtype, const void* cache,
                      int64_t n_pages, const int32_t* block_table, int64_t n_seqs,
                      int64_t max_blocks, const int32_t* seq_lens, const int32_t* q_start,
                      const awq_kv4_config* cfg, int64_t max_q, int64_t max_len, float scale,
                      int64_t window, void* out, float* lse_out, void* workspace,
                      size_t workspace_bytes, void* stream) {
  if (!q || !out) return AWQ_E_NULL;
  awq::Kv4Cache c;
  int st = kv4_cache(cache, n_pages, block_table, n_seqs, max_blocks, seq_lens, q_start, n_tokens,
                     cfg, &c);
  if (st) return st;
  if (!dtype_valid(dtype)) return AWQ_E_CONFIG;
  if (!(scale > 0.0f) || !(scale < __builtin_inff())) return AWQ_E_CONFIG;
  if (window < 0 || (st = attention_shape(n_tokens, n_seqs, heads, cfg, max_q, max_len)))
    return AWQ_E_SHAPE;
  if ((st = kv4_rows(q, q_token_stride, q_head_stride))) return st;
  if (!aligned(out, 16) || !aligned(lse_out, 4)) return AWQ_E_ALIGN;
  if (n_tokens == 0 || n_seqs == 0 || max_q == 0) return AWQ_OK;
  const awq::Kv4Plan p = awq::kv4_plan(n_seqs, (int)heads, cfg->kv_heads, cfg->head_dim,
                                       cfg->group_size, max_q, max_len, window);
  if (awq::kv4_blocks(p, (int)n_seqs, cfg->kv_heads) > awq::kMaxBlocks) return AWQ_E_SHAPE;
  // of this very plan, so that no launch can write past what it was given
  const size_t need =
      round_up(awq::kv4_workspace(p, n_tokens, n_seqs, (int)heads, cfg->kv_heads, cfg->head_dim), kAlign);
  if (need && (!workspace || workspace_bytes < need)) return AWQ_E_WORKSPACE;
  if (need && !aligned(workspace, kAlign)) return AWQ_E_ALIGN;
  if ((st = device_ptrs({q, cache, block_table, seq_lens, q_start, out, lse_out,
                         need ? workspace : nullptr})))
    return st;
  clear_pending_error();
  const awq::Kv4Query a{q, q_token_stride, q_head_stride, n_tokens, (int)heads, (int)max_q,
                        (int)max_len, (int)(window < (1 << 30) ? window : 0), scale,
                        dtype == AWQ_BF16, out, lse_out};
  return hip_status(awq::launch_kv4_attention(c, a, p, workspace, (hipStream_t)stream));
}

}  // extern "C"
