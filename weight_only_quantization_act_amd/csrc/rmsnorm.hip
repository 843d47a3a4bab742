// Root-mean-square norm with the residual's addition: h = x + r (rounded to the tokens' type), v =
// h w / sqrt(mean h^2 + eps), left as 16-bit values, as a row of 8-bit integers or as MXFP4.
//
// Pages: "AWQ" scholia-log notes §4.3 (S^-1 folded into the preceding operation: the norm's weight
// takes it), §2.3 (the quantiser of a row).
//
// Codes are decided at borders between values, so v is defined as the formula's value rounded to fp32
// once: squares of 16-bit values are exact in fp64 and summed there, the product h w (11 + 24 bits) is
// exact there, and v = fp32((h w) r) with r to within two ulp of fp64.  What of this is fp64 costs a few
// instructions a value at fp32's rate; the call is bound by memory: each value is read once (and the
// residual, and the sum written) and stays in registers between the sum and the rounding.  Rows too
// long for that are read a second time, from cache.  The 8-bit row's step needs the largest |v|:
// rounding is monotone, so it is that of max |h w|, found beside the sum.
#include <hip/hip_runtime.h>

#include "grid.h"
#include "int8_quant.h"
#include "mx_format.h"
#include "mx_internal.h"
#include "serve_internal.h"

namespace awq {

namespace {

// 8 columns of a 16-bit row as they lie in memory (0 past the last), and their values.
__device__ __forceinline__ uint4 raw8(const uint16_t* a, int c0, int K, bool vec) {
  if (vec && c0 + 8 <= K) return *(const uint4*)(a + c0);
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t lo = c0 + 2 * j < K ? a[c0 + 2 * j] : 0u, hi = c0 + 2 * j + 1 < K ? a[c0 + 2 * j + 1] : 0u;
    w[j] = lo | (hi << 16);
  }
  return uint4{w[0], w[1], w[2], w[3]};
}

template <bool BF16>
__device__ __forceinline__ void values8(const uint4& r, float (&v)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = from16<BF16>(w[j] & 0xffffu);
    v[2 * j + 1] = from16<BF16>(w[j] >> 16);
  }
}

template <bool BF16>
__device__ __forceinline__ void store8(uint16_t* a, int c0, int K, bool vec, const float (&v)[8]) {
  uint16_t o[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = to16<BF16>(v[j]);
  if (vec && c0 + 8 <= K) {
    uint4 p;
    p.x = o[0] | ((uint32_t)o[1] << 16);
    p.y = o[2] | ((uint32_t)o[3] << 16);
    p.z = o[4] | ((uint32_t)o[5] << 16);
    p.w = o[6] | ((uint32_t)o[7] << 16);
    *(uint4*)(a + c0) = p;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c0 + j < K) a[c0 + j] = o[j];
  }
}

template <bool BF16>
__device__ __forceinline__ void weight8(const NormArgs& a, int c0, bool vec, float (&w)[8]) {
  if (!a.w) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 1.0f;
  } else if (!a.w32) {
    values8<BF16>(raw8((const uint16_t*)a.w, c0, a.cols, vec), w);
  } else if (vec && c0 + 8 <= a.cols) {
    const float4 s0 = *(const float4*)((const float*)a.w + c0), s1 = *(const float4*)((const float*)a.w + c0 + 4);
    const float sv[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = sv[j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = c0 + j < a.cols ? ((const float*)a.w)[c0 + j] : 0.0f;
  }
}

// 1 / sqrt(x): the hardware's estimate e0 (relative error d, 2^-26 or so) and one step of third order,
// y = e0 (1 + d + 3/2 d^2 ...) with 2 d = 1 - x e0^2; NaN for an infinite x.
__device__ __forceinline__ double inverse_root(double x) {
  const double y = __builtin_amdgcn_rsq(x);
  const double e = fma(-(x * y), y, 1.0);
  return fma(y * e, fma(e, 0.375, 0.5), y);
}

// WPR waves a row; NCH 8-column chunks a thread in registers (0: the row is read twice).
template <bool BF16, int OUT, int WPR, int NCH>
__global__ __launch_bounds__(WPR == 1 ? 256 : 64 * WPR) void k_rmsnorm(NormArgs a, unsigned vec_mask) {
  __shared__ double red[2][WPR == 1 ? 1 : WPR];
  constexpr int kThreads = 64 * WPR;
  const int tid = WPR == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t row = WPR == 1 ? (int64_t)block_number() * 4 + (threadIdx.x >> 6) : (int64_t)block_number();
  if (row >= a.rows) return;  // the whole wave, or block
  const bool vx = vec_mask & 1, vr = vec_mask & 2, vh = vec_mask & 4, vw = vec_mask & 8, vy = vec_mask & 16;
  const int K = a.cols;
  // 8-column chunks: whole 16-byte groups of codes, whole words of scales
  const int nch = OUT == kNormMxfp4 ? (K + 127) / 128 * 16 : OUT == kNormInt8 ? (K + 15) / 16 * 2 : (K + 7) / 8;
  const uint16_t* x = a.x + row * a.ldx;
  const uint16_t* r = a.r ? a.r + row * a.ldr : nullptr;
  uint16_t* hrow = a.r ? a.h + row * a.ldh : nullptr;

  double sum = 0.0, top = 0.0;
  // the sum of x and r, stored
  auto take = [&](int ch, const uint4& xv, const uint4& rv, float (&h)[8]) {
    values8<BF16>(xv, h);
    if (r) {
      float t[8];
      values8<BF16>(rv, t);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = from16<BF16>(to16<BF16>(h[j] + t[j]));
      store8<BF16>(hrow, 8 * ch, K, vh, h);
    }
  };
  auto add = [&](int ch, const float (&h)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fma((double)h[j], (double)h[j], sum);
    if constexpr (OUT == kNormInt8) {
      float w[8];
      weight8<BF16>(a, 8 * ch, vw, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double p = (double)h[j] * (double)w[j];
        top = fmax(top, fabs(p));
        sum = fma(p, 0.0, sum);  // an infinite or NaN weight makes the row NaN
      }
    }
  };
  float h[NCH > 0 ? NCH : 1][8];
  if constexpr (NCH > 0) {
    // all loads before the first store (h may be x or r themselves)
    uint4 xv[NCH], rv[NCH];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int ch = tid + c * kThreads;
      if (ch < nch) {
        xv[c] = raw8(x, 8 * ch, K, vx);
        rv[c] = r ? raw8(r, 8 * ch, K, vr) : uint4{0, 0, 0, 0};
      }
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int ch = tid + c * kThreads;
      if (ch < nch) {
        take(ch, xv[c], rv[c], h[c]);
        add(ch, h[c]);
      }
    }
  } else {
    for (int ch = tid; ch < nch; ch += kThreads) {
      take(ch, raw8(x, 8 * ch, K, vx), r ? raw8(r, 8 * ch, K, vr) : uint4{0, 0, 0, 0}, h[0]);
      add(ch, h[0]);
    }
  }

#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    sum += __shfl_xor(sum, off);
    if constexpr (OUT == kNormInt8) top = fmax(top, __shfl_xor(top, off));
  }
  if constexpr (WPR > 1) {
    const int wave = threadIdx.x >> 6;
    if ((tid & 63) == 0) {
      red[0][wave] = sum;
      if constexpr (OUT == kNormInt8) red[1][wave] = top;
    }
    __syncthreads();
    sum = red[0][0];
    if constexpr (OUT == kNormInt8) top = red[1][0];
#pragma unroll
    for (int w = 1; w < WPR; ++w) {
      sum += red[0][w];
      if constexpr (OUT == kNormInt8) top = fmax(top, red[1][w]);
    }
  }
  const double inv = inverse_root(fma(sum, a.inv_cols, a.eps));

  RowStep st;
  if constexpr (OUT == kNormInt8) {
    // top and inv are at least 0 or inv is NaN
    st = row_step(__builtin_bit_cast(uint32_t, (float)(top * inv)) & 0x7fffffffu);
    if (tid == 0) ((float*)a.scales)[row] = st.step;
  }
  auto write = [&](int ch, const float (&hc)[8]) {
    float w[8], v[8];
    weight8<BF16>(a, 8 * ch, vw, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (float)((double)hc[j] * (double)w[j] * inv);
    if constexpr (OUT == kNormSame) {
      store8<BF16>((uint16_t*)a.y + row * a.ldy, 8 * ch, K, vy, v);
    } else if constexpr (OUT == kNormInt8) {
      *(uint2*)((int8_t*)a.y + row * a.ldy + 8 * ch) = row_codes8(v, st);
    } else {
      if (8 * ch >= K) {  // blocks past the last are zeros in a row of NaN, too
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
      }
      uint32_t byte;
      const uint32_t c = mx_codes8(v, byte);
      if (ch < (K + 31) / 32 * 4) *(uint32_t*)((uint8_t*)a.y + row * a.ldy + 4 * ch) = c;
      const uint32_t word = mx_scale_word(byte);
      if ((ch & 15) == 0) ((uint32_t*)a.scales)[(int64_t)(ch >> 4) * a.ld_scales + row] = word;
    }
  };
  if constexpr (NCH > 0) {
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int ch = tid + c * kThreads;
      if (ch < nch) write(ch, h[c]);
    }
  } else {
    for (int ch = tid; ch < nch; ch += kThreads) {
      values8<BF16>(raw8(r ? hrow : x, 8 * ch, K, r ? vh : vx), h[0]);
      write(ch, h[0]);
    }
  }
}

template <bool BF16, int OUT>
hipError_t launch_out(const NormArgs& a, unsigned vec, hipStream_t stream) {
  const int nch = (a.cols + 127) / 128 * 16;
  const dim3 grid = grid_of(a.rows);
#define AWQ_NORM(W, N)                                                                              \
  hipLaunchKernelGGL((k_rmsnorm<BF16, OUT, W, N>), grid, dim3(64 * W), 0, stream, a, vec)
  if (nch <= 2 * 256) AWQ_NORM(4, 2);
  else if (nch <= 4 * 256) AWQ_NORM(4, 4);
  else if (nch <= 8 * 256) AWQ_NORM(4, 8);
  else AWQ_NORM(4, 0);
#undef AWQ_NORM
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t stream) {
  if (a.rows <= 0) return hipSuccess;
  auto rows16 = [](const void* p, int64_t ld) { return ((uintptr_t)p % 16) == 0 && ld % 8 == 0; };
  const unsigned vec = (rows16(a.x, a.ldx) ? 1 : 0) | (rows16(a.r, a.ldr) ? 2 : 0) |
                       (rows16(a.h, a.ldh) ? 4 : 0) | (((uintptr_t)a.w % 16) == 0 ? 8 : 0) |
                       (a.out == kNormSame && rows16(a.y, a.ldy) ? 16 : 0);
#define AWQ_NORM_OUT(B)                                                  \
  a.out == kNormSame   ? launch_out<B, kNormSame>(a, vec, stream)        \
  : a.out == kNormInt8 ? launch_out<B, kNormInt8>(a, vec, stream)        \
                       : launch_out<B, kNormMxfp4>(a, vec, stream)
  return a.bf16 ? (AWQ_NORM_OUT(true)) : (AWQ_NORM_OUT(false));
#undef AWQ_NORM_OUT
}

}  // namespace awq
