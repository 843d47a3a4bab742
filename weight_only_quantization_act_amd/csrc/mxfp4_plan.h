// How a product in MXFP4 is laid out, by its sizes (host code without HIP, so that it can be compiled
// and looked at by itself).
#pragma once

#include <stdint.h>

namespace awq {

enum { kMxFew, kMxTile32, kMxTile64, kMxTile128, kMxTile256 };  // tiles by their tokens
struct MxPlan {
  int form, splits;
};

// KB: bytes of codes a row (two columns a byte).
inline MxPlan mxfp4_plan(int64_t T, int64_t M, int64_t KB) {
  MxPlan p{kMxTile128, 1};
  auto tiles_of = [&](int64_t bt, int64_t bm) { return ((T + bt - 1) / bt) * ((M + bm - 1) / bm); };
  if (T <= 16) p.form = kMxFew;
  else if (T <= 32) p.form = kMxTile32;
  else if (T <= 128) p.form = kMxTile64;
  else if (tiles_of(256, 256) >= 200) p.form = kMxTile256;
  if (p.form < kMxTile32 || p.form == kMxTile256) return p;
  const int64_t tiles = tiles_of(p.form == kMxTile32 ? 32 : p.form == kMxTile64 ? 64 : 128, 128);
  // K split over two blocks a compute unit, at least eight steps a split
  int64_t s = 512 / tiles;
  const int64_t most = KB / 1024;
  if (s > most) s = most;
  if (s > 8) s = 8;
  p.splits = (int)(s < 1 ? 1 : s);
  return p;
}

// The weight-streaming form's outputs a block, in tiles of 16.
inline int mxfp4_few_rows(int64_t M) { return M >= 32 * 512 ? 2 : 1; }

}  // namespace awq
