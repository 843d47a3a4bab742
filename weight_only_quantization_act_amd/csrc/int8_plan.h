// How a product in 8-bit integers is laid out, by its sizes (host code without HIP, so that it can be
// compiled and looked at by itself).
#pragma once

#include <stdint.h>

namespace awq {

// How one product runs, by its sizes.
enum { kFew, kTile32, kTile64, kTile128, kTile256 };  // tiles by their tokens
struct Int8Plan {
  int form, splits;
};

// Which form: what each measured, in us at 4096 x 4096, 11008 x 4096, 5120 x 13824 (out x in):
//   up to 16 tokens  weight streaming 7.3, 14.8, 27.6; 32-token tiles 9.0, 14.6, 20.6 (so weights of
//                    2^26 bytes and more take those)
//   32 tokens        32-token tiles 9.7, 15.6, 21.1; 64-token tiles 11.0, 16.7, 21.7
//   128              64: 15.4, 22.0, 24.0; 128: 16.3, 22.9, 26.8
//   200              64: 20.3, 27.0, 33.8; 128: 19.7, 28.9, 37.8
//   512              64: 24.9, 44.5, 67.2; 128: 28.0, 41.1, 53.9
//   1024             64: 31.2, 79.2, 109; 128: 36.9, 72.0, 94.9; 256: 53.3, 63.8, 131
//   4096             128: 88.7, 233, 298; 256: 72.7, 196, 322
// 64-token tiles stay ahead while they are one round of two blocks a compute unit and the sums are
// short.  256 x 256 tiles do 1.3 times the work of 128 x 128 ones a unit of time, but one a compute
// unit: a round of them costs 1.53 rounds of the small ones, a round begun nearly as much as a whole.
// The limits lie between what was measured at these three shapes; elsewhere they are carried over.
inline Int8Plan int8_plan(int64_t T, int64_t M, int64_t K) {
  Int8Plan p{kTile128, 1};
  auto tiles_of = [&](int64_t bt, int64_t bm) { return ((T + bt - 1) / bt) * ((M + bm - 1) / bm); };
  if (T <= 16 && M * K < (int64_t)1 << 26) p.form = kFew;
  else if (T <= 32) p.form = kTile32;
  else if (T <= 128 || (K <= 6144 && tiles_of(64, 128) <= 512)) p.form = kTile64;
  else {
    const int64_t small = tiles_of(128, 128), large = tiles_of(256, 256);
    const double rs = small / 512.0, cs = (double)((small + 511) / 512);
    const double rl = large / 256.0, cl = (double)((large + 255) / 256);
    if (1.53 * (0.25 * rl + 0.75 * cl) < 0.5 * (rs + cs)) p.form = kTile256;
  }
  if (p.form < kTile32 || p.form == kTile256) return p;
  const int64_t tiles = tiles_of(p.form == kTile32 ? 32 : p.form == kTile64 ? 64 : 128, 128);
  // K split over two blocks a compute unit, at least eight steps a split (5120 x 13824, unsplit and
  // split: 64 tokens 41.5 and 23.4 us, 200 tokens 72.5 and 35.1, 512 tokens 75.3 and 55.3)
  int64_t s = 512 / tiles;
  const int64_t most = K / 1024;
  if (s > most) s = most;
  if (s > 8) s = 8;
  p.splits = (int)(s < 1 ? 1 : s);
  return p;
}

// The weight-streaming form's outputs a block, in tiles of 16: two where that still leaves two blocks a
// compute unit.
inline int few_rows(int64_t M) { return M >= 32 * 512 ? 2 : 1; }

}  // namespace awq
