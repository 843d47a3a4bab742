// Rows of MXFP4 from 16-bit rows (A, A / s or A * s) and back; read-back of 8-bit rows.
//
// Pages: "AWQ" scholia-log notes §2.3 (a group's range sets its step, values round to the grid), §4.3
// (S^-1 folded into the activations).  The format is the OCP microscaling one: see mx_format.h.
//
// Bound by memory: 2 bytes of every value in, 17/32 out.  A block takes 8 rows of 512 columns, each wave two
// of them, so that loads are 1 KiB in one piece and the fold's scales serve two rows; 16 rows, four a wave,
// where many rows are divided by scales and in both ways back.  28672 rows of 8192 times scales 101-121 us (595
// MB, 4.9-5.9 TB/s), divided by them 124-130 us (the vector instructions of the reciprocals), back 92-95 us;
// 8-bit rows of that size back 121 us (705 MB, 5.8 TB/s).
#include <hip/hip_runtime.h>

#include "grid.h"
#include "mx_format.h"
#include "mx_internal.h"
#include "serve_internal.h"

namespace awq {

namespace {

// Rows a block, in us at 4, 8, 16 and 32: 28672 of 8192 times scales 129, 120, 125, 131; read back 110, 99,
// 95, 110.  Divided by scales, where a block has their reciprocals to find first, and many rows 16: 28672 of
// 8192 at 8 and 16 158, 128, 4096 of 4096 11.4, 10.5, but 333 of 13824 5.2 both, 50 of 4096 2.9, 3.5.
constexpr int kRowsTile = 8, kDivideTile = 16, kValuesTile = 16;
constexpr int kTileWords = 4;  // scale words (128 columns) of a row a block

// FOLD: kFoldNone, kFoldDivide or kFoldMultiply.
template <bool BF16, int FOLD, int TILE>
__global__ __launch_bounds__(256) void k_mxfp4_rows(const uint16_t* __restrict__ A, unsigned rows,
                                                    int K, int64_t lda, const float* __restrict__ s,
                                                    uint8_t* __restrict__ codes, int64_t ldc,
                                                    uint32_t* __restrict__ scales, int64_t lds,
                                                    unsigned tiles_k) {
  constexpr int R = TILE / 4;  // rows a wave
  const unsigned b = block_number();
  const unsigned tr = b / tiles_k, tk = b - tr * tiles_k;
  if (tr * TILE >= rows) return;  // the whole block
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c0 = (int)(tk * (kTileWords * 128)) + 8 * lane;
  const int q = c0 >> 7;
  if (q >= (K + 127) >> 7) return;  // sixteen lanes together; no barrier follows
  const bool stored = c0 < (K + 31) / 32 * 32;
  const unsigned row0 = tr * TILE + R * wave;
  // all rows' loads before the first is used; rows past the last repeat it
  u32x4 raw[R];
#pragma unroll
  for (int i = 0; i < R; ++i) raw[i] = raw8(A + (int64_t)min(row0 + i, rows - 1) * lda, c0, K);
  float sv[8];
  if constexpr (FOLD != kFoldNone) floats8(s, c0, K, 1.0f, sv);
  double inv[8];
  if constexpr (FOLD == kFoldDivide) {
#pragma unroll
    for (int j = 0; j < 8; ++j) inv[j] = reciprocal(sv[j]);
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const unsigned row = row0 + i;
    if (row >= rows) return;  // the whole wave
    float v[8];
    values8<BF16>(raw[i], v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (FOLD == kFoldMultiply) v[j] = v[j] * sv[j];
      if constexpr (FOLD == kFoldDivide) v[j] = (float)((double)v[j] * inv[j]);
    }
    uint32_t byte;
    const uint32_t c = mx_codes8(v, byte);
    if (stored) *(uint32_t*)(codes + (int64_t)row * ldc + (c0 >> 1)) = c;
    const uint32_t w = mx_scale_word(byte);
    if ((lane & 15) == 0) scales[(int64_t)q * lds + row] = w;
  }
}

template <bool BF16>
__global__ __launch_bounds__(256) void k_mxfp4_values(const uint8_t* __restrict__ codes, int64_t ldc,
                                                      const uint32_t* __restrict__ scales, int64_t lds,
                                                      unsigned rows, int K, uint16_t* __restrict__ out,
                                                      int64_t ldo, unsigned tiles_k) {
  const unsigned b = block_number();
  const unsigned tr = b / tiles_k, tk = b - tr * tiles_k;
  if (tr * kValuesTile >= rows) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c0 = (int)(tk * (kTileWords * 128)) + 8 * lane;
  if (c0 >= K) return;
#pragma unroll
  for (int i = 0; i < kValuesTile / 4; ++i) {
    const unsigned row = tr * kValuesTile + 4 * i + wave;
    if (row >= rows) return;
    const uint32_t c = *(const uint32_t*)(codes + (int64_t)row * ldc + (c0 >> 1));
    const uint32_t word = scales[(int64_t)(c0 >> 7) * lds + row];
    const uint32_t byte = (word >> (8 * ((c0 >> 5) & 3))) & 255u;
    const float sc = byte == 255 ? __builtin_nanf("") : mx_scale(byte);
    typedef float f2 __attribute__((ext_vector_type(2)));
    const f2 e[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, sc, 0),
                     __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, sc, 1),
                     __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, sc, 2),
                     __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, sc, 3)};
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = e[j >> 1][j & 1];
    store8(out + (int64_t)row * ldo, c0, K, pack8<BF16>(v));
  }
}

template <bool BF16>
__global__ __launch_bounds__(256) void k_int8_values(const int8_t* __restrict__ codes, int64_t ldc,
                                                     const float* __restrict__ steps, unsigned rows,
                                                     int K, uint16_t* __restrict__ out, int64_t ldo,
                                                     unsigned tiles_k) {
  const unsigned b = block_number();
  const unsigned tr = b / tiles_k, tk = b - tr * tiles_k;
  if (tr * kValuesTile >= rows) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c0 = (int)(tk * (kTileWords * 128)) + 8 * lane;
  if (c0 >= K) return;
#pragma unroll
  for (int i = 0; i < kValuesTile / 4; ++i) {
    const unsigned row = tr * kValuesTile + 4 * i + wave;
    if (row >= rows) return;
    const uint2 c = *(const uint2*)(codes + (int64_t)row * ldc + c0);
    const float st = steps[row];
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = (float)(int8_t)(c.x >> (8 * j)) * st;
      v[j + 4] = (float)(int8_t)(c.y >> (8 * j)) * st;
    }
    // the product is an fp32 number before it is rounded to the type: product and conversion would
    // otherwise become one instruction that rounds once
#pragma unroll
    for (int j = 0; j < 8; ++j) asm volatile("" : "+v"(v[j]));
    store8(out + (int64_t)row * ldo, c0, K, pack8<BF16>(v));
  }
}

int64_t tiles(int64_t rows, int64_t cols, int tile) {
  return (rows + tile - 1) / tile * ((cols + kTileWords * 128 - 1) / (kTileWords * 128));
}
unsigned col_tiles(int cols) { return (unsigned)((cols + kTileWords * 128 - 1) / (kTileWords * 128)); }

}  // namespace

// (at most: the largest of its forms)
int64_t mxfp4_rows_blocks(int64_t rows, int64_t cols) { return tiles(rows, cols, kRowsTile); }
int64_t values_blocks(int64_t rows, int64_t cols) { return tiles(rows, cols, kValuesTile); }

hipError_t launch_mxfp4_rows(const void* A, int64_t rows, int cols, int64_t lda, bool bf16,
                             const float* s, int fold, uint8_t* codes, int64_t ld_codes,
                             uint32_t* scales, int64_t ld_scales, hipStream_t stream) {
  if (rows <= 0 || cols <= 0) return hipSuccess;
  const int f = s ? fold : kFoldNone;
  const bool many = tiles(rows, cols, kDivideTile) >= 1024;  // (four blocks a compute unit)
#define AWQ_MXROWS(B, F, TILE)                                                               \
  hipLaunchKernelGGL((k_mxfp4_rows<B, F, TILE>), grid_of(tiles(rows, cols, TILE)), dim3(256), 0, stream, \
                     (const uint16_t*)A, (unsigned)rows, cols, lda, s, codes, ld_codes, scales, \
                     ld_scales, col_tiles(cols))
#define AWQ_MXROWS_F(B)                                                    \
  if (f == kFoldNone) AWQ_MXROWS(B, kFoldNone, kRowsTile);                 \
  else if (f == kFoldMultiply) AWQ_MXROWS(B, kFoldMultiply, kRowsTile);    \
  else if (many) AWQ_MXROWS(B, kFoldDivide, kDivideTile);                  \
  else AWQ_MXROWS(B, kFoldDivide, kRowsTile)
  if (bf16) {
    AWQ_MXROWS_F(true);
  } else {
    AWQ_MXROWS_F(false);
  }
#undef AWQ_MXROWS_F
#undef AWQ_MXROWS
  return hipGetLastError();
}

hipError_t launch_mxfp4_values(const uint8_t* codes, int64_t ld_codes, const uint32_t* scales,
                               int64_t ld_scales, int64_t rows, int cols, bool bf16, void* out,
                               int64_t ldo, hipStream_t stream) {
  if (rows <= 0 || cols <= 0) return hipSuccess;
  const dim3 grid = grid_of(values_blocks(rows, cols));
  if (bf16)
    hipLaunchKernelGGL((k_mxfp4_values<true>), grid, dim3(256), 0, stream, codes, ld_codes, scales,
                       ld_scales, (unsigned)rows, cols, (uint16_t*)out, ldo, col_tiles(cols));
  else
    hipLaunchKernelGGL((k_mxfp4_values<false>), grid, dim3(256), 0, stream, codes, ld_codes, scales,
                       ld_scales, (unsigned)rows, cols, (uint16_t*)out, ldo, col_tiles(cols));
  return hipGetLastError();
}

hipError_t launch_int8_values(const int8_t* codes, int64_t ld_codes, const float* steps, int64_t rows,
                              int cols, bool bf16, void* out, int64_t ldo, hipStream_t stream) {
  if (rows <= 0 || cols <= 0) return hipSuccess;
  const dim3 grid = grid_of(values_blocks(rows, cols));
  if (bf16)
    hipLaunchKernelGGL((k_int8_values<true>), grid, dim3(256), 0, stream, codes, ld_codes, steps,
                       (unsigned)rows, cols, (uint16_t*)out, ldo, col_tiles(cols));
  else
    hipLaunchKernelGGL((k_int8_values<false>), grid, dim3(256), 0, stream, codes, ld_codes, steps,
                       (unsigned)rows, cols, (uint16_t*)out, ldo, col_tiles(cols));
  return hipGetLastError();
}

}  // namespace awq
