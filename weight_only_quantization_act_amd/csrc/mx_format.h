// Microscaled 4-bit floating point (MXFP4), device side: blocks of 32 columns share a power of two
// 2^(b - 127) with one byte b (255: NaN), an element is a sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6.
//
// A lane holds 8 consecutive columns, a block is four lanes of a quad, the 128 columns whose four scale
// bytes share a 32-bit word are sixteen lanes of a row.  With e the exponent field of the
// block's largest magnitude, floor(log2) + 127, the scale is b = max(e, 2) - 2: the largest magnitude
// over the scale lies in [4, 8) (below 4 where b is 0) and the elements round to nearest, ties to even,
// and saturate at 6, as v_cvt_scalef32_pk_fp4_f32 does, subnormal scales included (checked on the
// device against the formula for all ties and their neighbours at every scale).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "int8_quant.h"
#include "quantizer.h"

#pragma clang fp contract(off)

namespace awq {

// Columns [c0, c0 + 8) of a 16-bit row as they lie in memory, zeros from K on; their values; such
// values stored; 8 of a vector of fp32, `fill` from K on.  Rows begin at any even address: a global
// load or store of 16 bytes takes every alignment on this target.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef f32x4 f32x4_at4 __attribute__((aligned(4)));

__device__ __forceinline__ u32x4 raw8(const uint16_t* a, int c0, int K) {
  if (c0 + 8 <= K) return *(const u32x4_at2*)(a + c0);
  uint32_t h[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) h[j] = a[min(c0 + j, K - 1)];
#pragma unroll
  for (int j = 0; j < 8; ++j) h[j] = c0 + j < K ? h[j] : 0u;
  return u32x4{h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16)};
}

template <bool BF16>
__device__ __forceinline__ void values8(const u32x4& r, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t w = r[j];
    v[2 * j] = from16<BF16>(w & 0xffffu);
    v[2 * j + 1] = from16<BF16>(w >> 16);
  }
}

template <bool BF16>
__device__ __forceinline__ u32x4 pack8(const float (&v)[8]) {
  u32x4 r;
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = to16<BF16>(v[2 * j]) | ((uint32_t)to16<BF16>(v[2 * j + 1]) << 16);
  return r;
}

__device__ __forceinline__ void store8(uint16_t* a, int c0, int K, const u32x4& r) {
  if (c0 + 8 <= K) {
    *(u32x4_at2*)(a + c0) = r;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c0 + j < K) a[c0 + j] = (uint16_t)(r[j >> 1] >> (16 * (j & 1)));
  }
}

__device__ __forceinline__ void floats8(const float* a, int c0, int K, float fill, float (&v)[8]) {
  if (c0 + 8 <= K) {
    const f32x4 lo = *(const f32x4_at4*)(a + c0), hi = *(const f32x4_at4*)(a + c0 + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = lo[j];
      v[j + 4] = hi[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = a[min(c0 + j, K - 1)];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c0 + j < K ? v[j] : fill;
  }
}

// 1 / s in fp64, to within 2^-52 of itself: the hardware's estimate y and a step of third order, 1/s = y (1 + e
// + e^2 ...) with e = 1 - s y.  (1 / inf is y, a zero; of a zero it is NaN in place of an infinity, which
// makes no difference to a block.)
//
// A 16-bit value v times it, rounded to fp32, is v / s rounded correctly: a border between two fp32
// numbers is M 2^k with an odd M of 25 bits, s = S 2^l with S below 2^24 and v an integer of 11 bits times a
// power of two, so v - s M 2^k is a multiple of a unit that s M 2^k holds less than 2^49 times, and not 0; v / s
// lies 2^-49 or more of itself from every border, the product less than 2^-51 from v / s.  (Where the
// result is subnormal a tie can be exact and come out either way; it is then an odd number of 11 bits times
// 2^-150, which is far below the least element's border, 2^-129.)
__device__ __forceinline__ double reciprocal(float s) {
  const double d = (double)s, y = __builtin_amdgcn_rcp(d);
  const double e = fma(-d, y, 1.0);
  const double r = fma(y, fma(e, e, e), y);
  return fabsf(s) == __builtin_inff() ? y : r;
}

__device__ __forceinline__ uint32_t quad_max_u32(uint32_t x) {
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, kDppQuadXor1, 0xf, 0xf, false));
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, kDppQuadXor2, 0xf, 0xf, false));
  return x;
}

// The scale byte of a block whose largest magnitude has these fp32 bits (infinities and NaN lie above
// all finite ones).
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
  return top >= 0x7f800000u ? 255u : max(top >> 23, 2u) - 2u;
}

// 2^(b - 127), b below 255
__device__ __forceinline__ float mx_scale(uint32_t b) {
  return __builtin_bit_cast(float, b == 0 ? 0x00400000u : b << 23);
}

// The lane's 8 codes, column 0 in the low nibble, and its block's scale byte.
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8], uint32_t& byte) {
  // (maxima that keep a NaN; one instruction for three values)
  float m = __builtin_elementwise_maximum(fabsf(v[0]), fabsf(v[1]));
#pragma unroll
  for (int j = 2; j < 8; ++j) m = __builtin_elementwise_maximum(m, fabsf(v[j]));
  byte = mx_scale_byte(quad_max_u32(__builtin_bit_cast(uint32_t, m) & 0x7fffffffu));
  const float sc = mx_scale(byte);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], sc, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], sc, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], sc, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], sc, 3);
  return byte == 255 ? 0u : c;
}

// The 32-bit word of a row's four scale bytes, in all of the sixteen lanes that hold them.
__device__ __forceinline__ uint32_t mx_scale_word(uint32_t byte) {
  uint32_t w = byte << (8 * ((threadIdx.x >> 2) & 3));
  w |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, 0x124, 0xf, 0xf, false);  // row_ror:4
  w |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, 0x128, 0xf, 0xf, false);  // row_ror:8
  return w;
}

}  // namespace awq
