// Device side of the 4-bit key/value cache: which sequence and position a row is, where its
// page lies.  The record layout is described in awq_serve.h; it is the order in which the
// attention's matrix instructions take their operands, so that a lane reads its words with
// 16-byte loads and a 16-bit half always belongs to one token (a token is written without
// reading its neighbours).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "serve_internal.h"

namespace awq {

// The sequence of row t (the last b with starts[b] <= t), or -1 past the last row.  A decode
// step has one row a sequence, so sequence t is tried before the search.
__device__ __forceinline__ int kv4_sequence(const Kv4Cache& c, int64_t t) {
  if (t < c.n_seqs && c.starts[t] == t && c.starts[t + 1] == t + 1) return (int)t;
  if (t >= c.starts[c.n_seqs]) return -1;
  int lo = 0, hi = c.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (c.starts[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Byte offset in the cache of the record that holds token pos of sequence b for a head, or -1
// where there is no such page.
__device__ __forceinline__ int64_t kv4_record_at(const Kv4Cache& c, int b, int pos, int head) {
  if (pos < 0) return -1;
  const int blk = pos >> c.log2p;
  if (blk >= c.max_blocks) return -1;
  const int page = c.table[(int64_t)b * c.max_blocks + blk];
  if (page < 0 || page >= c.n_pages) return -1;
  return ((int64_t)page * c.kv_heads + head) * c.record;
}

}  // namespace awq
