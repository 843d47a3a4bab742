// Grids of more blocks than one dimension takes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace awq {

// A dimension of a grid holds less than 2^32 threads (a launch of more loses blocks without an error):
// blocks, up to 2^31, in rows of 2^20.  Those past the end in the last row have nothing to do.
constexpr int kGridRowLog2 = 20;
inline dim3 grid_of(int64_t blocks) {
  constexpr int64_t kRow = (int64_t)1 << kGridRowLog2;
  return dim3((unsigned)(blocks < kRow ? blocks : kRow), (unsigned)((blocks + kRow - 1) / kRow));
}
// (of a constant row: the grid's own size would be a load before anything else)
__device__ __forceinline__ unsigned block_number() { return blockIdx.x + (blockIdx.y << kGridRowLog2); }

}  // namespace awq
