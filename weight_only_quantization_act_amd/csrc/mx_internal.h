// Launchers of the MXFP4 operators and of the norm, shared between their HIP files and the C-ABI layer.
// Every launcher enqueues on `stream` and returns the hipError_t of its launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace awq {

// MXFP4 rows: codes [rows][ld bytes], scales [columns / 128][ld_scales][4].
constexpr int64_t kMxMaxRows = ((int64_t)1 << 29) - 512;  // two rows of scales span less than 2^32 bytes
constexpr int64_t kMxMaxK = (int64_t)1 << 22;
constexpr int64_t kCacheBytes = 256 << 20;  // the last-level cache
inline int64_t mx_code_bytes(int64_t cols) { return (cols + 31) / 32 * 16; }
inline int64_t mx_words(int64_t cols) { return (cols + 127) / 128; }  // scale words of a row

hipError_t launch_mxfp4_rows(const void* A, int64_t rows, int cols, int64_t lda, bool bf16,
                             const float* s, int fold, uint8_t* codes, int64_t ld_codes,
                             uint32_t* scales, int64_t ld_scales, hipStream_t stream);
hipError_t launch_mxfp4_values(const uint8_t* codes, int64_t ld_codes, const uint32_t* scales,
                               int64_t ld_scales, int64_t rows, int cols, bool bf16, void* out,
                               int64_t ldo, hipStream_t stream);
hipError_t launch_int8_values(const int8_t* codes, int64_t ld_codes, const float* steps, int64_t rows,
                              int cols, bool bf16, void* out, int64_t ldo, hipStream_t stream);
// Blocks of these launches.
int64_t mxfp4_rows_blocks(int64_t rows, int64_t cols);
int64_t values_blocks(int64_t rows, int64_t cols);

// ---- product -----------------------------------------------------------------------------
struct MxArgs {
  const uint8_t* x;
  int64_t ldx;
  const uint32_t* xs;
  int64_t ldxs;
  const uint8_t* w;
  int64_t ldw;
  const uint32_t* ws;
  int64_t ldws;
  const void* bias;
  void* y;
  int64_t ldy;
  int T, M, KB;  // KB: bytes of codes a row that are read, a multiple of 16
  bool bf16;
};
hipError_t launch_mxfp4_matmul(const MxArgs& a, hipStream_t stream);
// The linear layer of few tokens in one launch: a.x and a.xs unused, x 16-bit with `cols` columns
// and row stride ldx.  Taken where mxfp4_linear_fused says so.
bool mxfp4_linear_fused(int64_t T, int64_t M, int64_t cols);
hipError_t launch_mxfp4_linear_fused(const MxArgs& a, const void* x, int64_t ldx, const float* s,
                                     int cols, hipStream_t stream);

// ---- norm --------------------------------------------------------------------------------
enum { kNormSame = 0, kNormInt8 = 1, kNormMxfp4 = 2 };
struct NormArgs {
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* r;  // residual, or NULL
  int64_t ldr;
  uint16_t* h;  // the sum (with r only)
  int64_t ldh;
  const void* w;  // 16-bit or fp32, or NULL: ones
  bool w32, bf16;
  double eps, inv_cols;  // inv_cols: 1 / cols
  int64_t rows;
  int cols;
  int out;  // kNorm...
  void* y;  // values or codes
  int64_t ldy;
  void* scales;  // int8: steps; mxfp4: scale words
  int64_t ld_scales;
};
hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t stream);

}  // namespace awq
