// Device side of the 8-bit row quantiser: loads with the fold of the scales, the row's
// largest magnitude, its step and the codes (see int8_rows.hip).  Every operation is a single
// IEEE fp32 operation without contraction, so the codes are the same in every kernel that
// forms them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "quantizer.h"
#include "serve_internal.h"

#pragma clang fp contract(off)

namespace awq {

// 16-byte loads of a row's 8-column chunks need the base, the row stride and s aligned.
inline bool row_vector_loads(const void* A, int64_t lda, const float* s) {
  return ((uintptr_t)A % 16) == 0 && lda % 8 == 0 && ((uintptr_t)s % 16) == 0;
}

template <bool BF16>
__device__ __forceinline__ float from16(uint32_t h) {
  if constexpr (BF16) return __builtin_bit_cast(float, h << 16);
  return h2f((uint16_t)h);
}

template <bool BF16>
__device__ __forceinline__ uint16_t to16(float f) {
  if constexpr (BF16) return __builtin_bit_cast(uint16_t, (__bf16)f);
  return f2h(f);
}

// v = the row's columns [c0, c0 + 8) after the fold; columns at or past K are 0.
template <bool BF16, bool VEC>
__device__ __forceinline__ void load_row8(const uint16_t* __restrict__ a,
                                          const float* __restrict__ s, int fold, int c0, int K,
                                          float (&v)[8]) {
  if (VEC && c0 + 8 <= K) {
    const uint4 r = *(const uint4*)(a + c0);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = from16<BF16>(w[j] & 0xffffu);
      v[2 * j + 1] = from16<BF16>(w[j] >> 16);
    }
    if (fold != kFoldNone) {
      const float4 s0 = *(const float4*)(s + c0), s1 = *(const float4*)(s + c0 + 4);
      const float sv[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = fold == kFoldDivide ? v[j] / sv[j] : v[j] * sv[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = 0.0f;
      if (c0 + j < K) {
        v[j] = from16<BF16>(a[c0 + j]);
        if (fold == kFoldDivide) v[j] = v[j] / s[c0 + j];
        if (fold == kFoldMultiply) v[j] = v[j] * s[c0 + j];
      }
    }
  }
}

// The largest magnitude as its bit pattern: for fp32 patterns without the sign, integer order
// is the order of the values, with infinity and then every NaN above all finite ones.
__device__ __forceinline__ uint32_t max_abs8(const float (&v)[8], uint32_t top) {
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, __builtin_bit_cast(uint32_t, v[j]) & 0x7fffffffu);
  return top;
}

template <int WAVES>
__device__ __forceinline__ uint32_t block_max(uint32_t top, uint32_t* red) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
  __syncthreads();
  top = red[0];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) top = max(top, red[w]);
  return top;
}

struct RowStep {
  float step, inv;
  bool finite;
};

__device__ __forceinline__ RowStep row_step(uint32_t top) {
  RowStep r;
  r.finite = top < 0x7f800000u;
  float st = __builtin_bit_cast(float, top) / 127.0f;
  if (st == 0.0f) st = 1.0f;
  r.inv = step_reciprocal(st);
  r.step = r.finite ? st : __builtin_nanf("");
  return r;
}

// The 8 codes of a chunk, low byte first.  rint(fl(v / step)) is taken as rint(fl(v * inv))
// with the hardware reciprocal (relative error <= 2^-23 for a normal step): |v / step| is at
// most 127 (1 + 2^-24), so fl(v * inv) lies within 127 * 3 * 2^-24 < 2^-15.3 of the exact
// quotient and fl(v / step) within 127 * 2^-24; unless the product is within 2^-14 of a
// half-integer both round to the same integer.  Inside that band, and for a step without a
// normal reciprocal, the correctly rounded division decides.  The clamp to [-127, 127] acts
// only where the step is subnormal (its own rounding can then be half of it).
__device__ __forceinline__ uint2 row_codes8(const float (&v)[8], const RowStep& r) {
  constexpr float kBand = 6.103515625e-05f;  // 2^-14
  float q[8];
  bool any = false, near[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float t = v[j] * r.inv;
    q[j] = rintf(t);
    near[j] = !(fabsf(fabsf(t - q[j]) - 0.5f) > kBand);
    any |= near[j];
  }
  if (any) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (near[j]) q[j] = rintf(v[j] / r.step);
  }
  uint2 o = {0u, 0u};
  if (r.finite) {
    int c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = (int)fminf(fmaxf(q[j], -127.0f), 127.0f) & 0xff;
    o.x = (uint32_t)(c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24));
    o.y = (uint32_t)(c[4] | (c[5] << 8) | (c[6] << 16) | (c[7] << 24));
  }
  return o;
}

}  // namespace awq
