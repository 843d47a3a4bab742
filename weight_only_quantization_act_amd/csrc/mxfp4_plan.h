// How a product in MXFP4 is laid out, by its sizes (host code without HIP, so that it can be compiled
// and looked at by itself).
#pragma once

#include <stdint.h>

namespace awq {

// Weights streamed through registers (few tokens); tiles by tokens x outputs, "K" with groups of waves that
// share the columns, "W" in more stages with one block a compute unit.
enum { kMxFew, kMxTile32K, kMxTile32x64K, kMxTile64K, kMxTile64, kMxTile64x128, kMxTile128W,
       kMxTile128, kMxTile256 };

// KB: bytes of codes a row (two columns a byte).
//
// Few: blocks of 16 outputs, one or two a compute unit, while what each reads stays small: its weights (as
// much as 16 tokens) and all tokens' operands.  Measured, streaming and the best tiles, in us (weights in
// the last-level cache):
//   tokens              1         8         16        32
//   4096 x 4096         4.1, 5.4  4.6, 5.9  4.9, 6.0  5.9, 5.9
//   4096 x 11008        6.5, 7.7  7.3, 7.8  8.2, 7.9  10.8, 7.9
//   2048 x 8192         5.2, 6.7            6.5, 6.9  8.4, 7.0
//   6144 x 4096                   5.9, 5.9  6.5, 6.0  8.5, 6.0
//   8192 x 3584                   5.5, 5.9  6.1, 6.0  7.9, 6.1
//   8192 x 8192                   9.8, 7.7  11.2, 8.1 15.0, 8.7
//   11008 x 4096        6.8, 6.3            8.4, 6.4  11.4, 6.4
// One token's limit past 4096 outputs is larger: its linear layer saves a launch where the product streams. The
// product, streamed and tiles, and the linear layer with scales, in one launch and in two with tiles (other
// weights each call):
//   5120 x 4096         5.8, 6.1  6.7, 8.3        8192 x 7744         9.4, 9.7  11.3, 12.4
//   5120 x 7744         8.6, 8.3  10.6, 11.0      past it: 5120 x 8192 9.4, 8.1  12.0, 10.4
//   6144 x 7744         8.8, 8.7  10.8, 11.3               8192 x 8192 9.8, 10.2 14.3, 12.6
//
// Tiles: the form with the smallest time a step of 256 columns, fitted to measurements (us a step at r
// tiles a compute unit; small tiles are bound by what goes through LDS, 128 x 128 ones run in rounds of two
// a compute unit, 256 x 256 ones of one):
//   tiles of 64 x 64    0.22-0.28 up to r = 1, 0.56 at 2, 0.68 at 2.7, 2.4 at 10.8
//            64 x 128   0.30-0.36 up to r = 1, 0.7 at 1.3, 1.15 at 2.7, 2.2 at 5.4
//            128 x 128  0.38-0.44 up to r = 1 in three stages (0.56-0.7 in two), 0.94-1.1 at 1 to 1.3,
//                       1.95 at 2 to 2.7 in two stages
//            256 x 256  1.4-1.5 up to r = 1, 1.8-2.0 a round beyond
// Between neighbours, in us, 64 x 64, 64 x 128, 128 x 128, 256 x 256: 333 tokens of 5120 x 13824 24.2,
// 22.0, 24.5, 69; 512 of it 35.3, 36.4, 25.7, 70; 512 of 11008 x 4096 24.5, 21.5, 20.4, 26.8; 1024 of
// 11008 x 4096 43, 40, 33.4, 30.1; 4096 of 11008 x 4096 165, 145, 109, 97.
// Where tiles leave at most one a compute unit, groups of waves share the columns of one (17 tokens of
// 5120 x 13824 on 64 x 64: one group 16.8, two 13.0) and the smallest tiles that fit are the fastest: 16
// tokens of 5120 x 13824 on 32 x 32 in four groups 9.3, 32 x 64 in two 11.7, 64 x 64 in two 12.8; 50 of
// 4096 x 4096 5.6, 6.4, 6.7; with more than one a unit they are not (50 of 11008 x 4096 12.6, 8.7, 7.1; 100
// of it 64 x 64 in two groups 12.4, one 9.6).
inline int mxfp4_form(int64_t T, int64_t M, int64_t KB) {
  if (T <= 32 && M <= 8192 && KB * (T + 16) <= (M <= 4096 ? 150000 : T == 1 ? 66000 : 54000)) return kMxFew;
  auto per_unit = [&](int64_t bt, int64_t bm) {
    return (double)(((T + bt - 1) / bt) * ((M + bm - 1) / bm)) / 256.0;
  };
  auto rounds = [](double r) { return (double)(int64_t)(r + 0.999999); };
  if (per_unit(32, 32) <= 1) return kMxTile32K;
  if (per_unit(32, 64) <= 1) return kMxTile32x64K;
  const double r1 = per_unit(64, 64), r2 = per_unit(64, 128), r3 = per_unit(128, 128), r4 = per_unit(256, 256);
  const double t1 = r1 <= 1 ? 0.27 : 0.1 + 0.24 * r1;
  const double t2 = r2 <= 1 ? 0.36 : 0.15 + 0.4 * r2;
  const double t3 = r3 <= 1 ? 0.42 : r3 <= 2 ? 0.95 : 1.05 * rounds(r3 / 2);
  const double t4 = r4 <= 1 ? 1.45 : 1.95 * rounds(r4);
  if (t1 <= t2 && t1 <= t3 && t1 <= t4) return r1 <= 1 ? kMxTile64K : kMxTile64;
  if (t2 <= t3 && t2 <= t4) return kMxTile64x128;
  if (t3 <= t4) return r3 <= 1 ? kMxTile128W : kMxTile128;
  return kMxTile256;
}

}  // namespace awq
