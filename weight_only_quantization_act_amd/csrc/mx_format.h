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

#include "quantizer.h"

#pragma clang fp contract(off)

namespace awq {

constexpr int kMxBlock = 32;

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
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, __builtin_bit_cast(uint32_t, v[j]) & 0x7fffffffu);
  byte = mx_scale_byte(quad_max_u32(top));
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
