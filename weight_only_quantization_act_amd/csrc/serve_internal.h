// Launchers of the serving operators, shared between their HIP files and the C-ABI layer.
// Every launcher enqueues on `stream` and returns the hipError_t of its launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace awq {

// Blocks of one launch at most: numbered in 32 bits, with a row of the grid to spare (grid.h).
constexpr int64_t kMaxBlocks = 0x7fffffff - (1 << 20);

// ---- rows of 8-bit integers ------------------------------------------------------------
constexpr int kFoldNone = -1, kFoldDivide = 0, kFoldMultiply = 1;
hipError_t launch_int8_rows(const void* A, int64_t rows, int cols, int64_t lda, bool bf16,
                            const float* s, int fold, int8_t* codes, int64_t ld_codes,
                            float* steps, hipStream_t stream);

// ---- product in 8-bit integers ---------------------------------------------------------
constexpr int64_t kInt8MaxK = 131056;  // 2^14 K stays below 2^31
struct Int8Args {
  const int8_t* x;
  int64_t ldx;
  const float* xstep;
  const int8_t* w;
  int64_t ldw;
  const float* wstep;
  const void* bias;
  void* y;
  int64_t ldy;
  int T, M, K;  // K: the bytes of a row that are read, a multiple of 16
  bool bf16;
};
size_t int8_matmul_workspace(int64_t T, int64_t M, int64_t K);
hipError_t launch_int8_matmul(const Int8Args& a, void* workspace, hipStream_t stream);
// The linear layer of one token in one launch: a.x, a.ldx and a.xstep unused, x 16-bit with
// `cols` columns.  Taken where int8_linear_fused says so.
bool int8_linear_fused(int64_t T, int64_t K);
hipError_t launch_int8_linear_fused(const Int8Args& a, const void* x, const float* s, int cols,
                                    hipStream_t stream);

// ---- key/value cache in 4 bits ---------------------------------------------------------
struct Kv4Cache {
  uint8_t* pages;
  int64_t n_pages;
  const int32_t* table;   // [n_seqs][max_blocks]
  const int32_t* lens;    // [n_seqs]
  const int32_t* starts;  // [n_seqs + 1]
  int n_seqs, max_blocks;
  int kv_heads, dim, group, log2p;
  int zero_point;
  unsigned record;  // bytes of one page of one head
};
inline unsigned kv4_record(int dim, int group, int page) {
  return (unsigned)page * dim + 8u * page * (dim / group);
}
// Blocks of a write or read-back: groups of 2048 / dim rows (see kv4_store.hip) for each key head.
constexpr int64_t kv4_store_blocks(int64_t n_tokens, int dim, int n_seqs, int kv_heads) {
  return (n_tokens / (2048 / dim) + 2 * n_seqs + 1) * kv_heads;
}
hipError_t launch_kv4_append(const Kv4Cache& c, const void* k, int64_t kt, int64_t kh,
                             const void* v, int64_t vt, int64_t vh, int64_t n_tokens, bool bf16,
                             hipStream_t stream);
hipError_t launch_kv4_read(const Kv4Cache& c, int64_t n_tokens, bool bf16, void* k, void* v,
                           hipStream_t stream);

struct Kv4Query {
  const void* q;
  int64_t qt, qh;  // token and head strides
  int64_t n_tokens;
  int heads, max_q, max_len, window;
  float scale;
  bool bf16;
  void* out;
  float* lse;
};
// How one attention call is laid out (by sizes only).  Columns are query rows x heads of a key
// head.
struct Kv4Plan {
  int wide;    // 0: up to 16 columns, a block's waves share the keys; 1: column tiles a wave
  int tiles;   // wide: blocks of columns a (sequence, key head)
  int splits;  // wide: parts of the keys; else blocks of a key head over which all keys are dealt
               // out.  1: none, otherwise a second launch joins the parts
  int waves;   // waves a block
};
Kv4Plan kv4_plan(int64_t n_seqs, int heads, int kv_heads, int dim, int group, int64_t max_q,
                 int64_t max_len, int64_t window);
inline int64_t kv4_blocks(const Kv4Plan& p, int n_seqs, int kv_heads) {
  return (int64_t)kv_heads * (p.wide ? (int64_t)p.tiles * p.splits * n_seqs : p.splits > 1 ? p.splits : n_seqs);
}
size_t kv4_workspace(const Kv4Plan& p, int64_t n_tokens, int64_t n_seqs, int heads, int kv_heads,
                     int dim);
// What covers the plan of every window.
size_t kv4_workspace_any_window(int64_t n_tokens, int64_t n_seqs, int heads, int kv_heads, int dim,
                                int group, int64_t max_q, int64_t max_len);
hipError_t launch_kv4_attention(const Kv4Cache& c, const Kv4Query& q, const Kv4Plan& p,
                                void* workspace, hipStream_t stream);

}  // namespace awq
