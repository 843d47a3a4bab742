// Launchers of the serving operators, shared between their HIP files and the C-ABI layer.
// Every launcher enqueues on `stream` and returns the hipError_t of its launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace awq {

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

}  // namespace awq
