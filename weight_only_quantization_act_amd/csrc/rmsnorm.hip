// Root-mean-square norm with the residual's addition: h = x + r (rounded to the tokens' type), v =
// h w / sqrt(mean h^2 + eps), left as 16-bit values, as a row of 8-bit integers or as MXFP4.
//
// Pages: "AWQ" scholia-log notes §4.3 (S^-1 folded into the preceding operation: the norm's weight
// takes it), §2.3 (the quantiser of a row).
//
// Codes are decided at borders between values, so v is the formula's value rounded to fp32 once, but for
// what fp64 leaves open: squares of 16-bit values are exact in fp64 and summed there, the product h w (11 +
// 24 bits) is exact there, and v = fp32((h w) r).  A thread adds its n squares one by one, n at most 32 or K /
// 512 + 8, so the sum lies within (n + 13) 2^-53 of itself, r, whose error is half of that and of the mean's two
// roundings, and the product within (n / 2 + 13) 2^-53 <= (K / 1024 + 29) 2^-53: only a value that close to the
// middle of two fp32 numbers can come out as the other one, and differ between forms.  What of this is fp64
// costs a few instructions a value at fp32's rate.  Each value is read once (and the residual, and the sum written)
// and stays in registers between the sum and the rounding; rows too long for that are read a second
// time, from cache.  Large calls are bound by memory (16384 rows of 8192 in bf16 with a residual to MXFP4
// 168 us, 877 MB at 5.2 TB/s), calls of a few thousand rows by their vector instructions and one
// pass of latencies (2047 rows of 5000 to MXFP4 11.4 us, 2.3 TB/s), few rows by the latencies alone (33 of
// 5120 to 8 bits 4.6 us, one of 4096 2.4 us).  The 8-bit row's step needs the largest |v|:
// rounding is monotone, so it is that of max |h w|, found beside the sum; these products and, again, the codes'
// bound many rows without a residual (16384 of 8192 with an fp32 weight 146 us of the 78 that the bytes
// take, vector units busy 89%; with a residual 186 of 182).
#include <hip/hip_runtime.h>

#include "grid.h"
#include "int8_quant.h"
#include "mx_format.h"
#include "mx_internal.h"
#include "serve_internal.h"

namespace awq {

namespace {

// The weights of 8 columns as they lie in memory: W32 fp32, else 16-bit (0 past the last column, 1 where
// there is no weight).
template <bool BF16, bool W32>
struct Weights {
  u32x4 r[W32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* w, int c0, int K) {
    if constexpr (W32) {
      float v[8];
      floats8((const float*)w, c0, K, 0.0f, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j >> 2][j & 3] = __builtin_bit_cast(uint32_t, v[j]);
    } else if (w) {
      r[0] = raw8((const uint16_t*)w, c0, K);
    } else {
      const uint32_t one = to16<BF16>(1.0f) * 0x10001u;
      r[0] = u32x4{one, one, one, one};
    }
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    if constexpr (W32) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t u = r[j >> 2][j & 3];
        v[j] = __builtin_bit_cast(float, u);
      }
    } else {
      values8<BF16>(r[0], v);
    }
  }
};

// The products of 8 fp16 values with 8 others, exact in fp32: one instruction from the packed halves (the
// third operand is -0, which keeps the sign of a product of 0).  Conversions are most of the norm's vector
// instructions: 2047 rows of 5000 to MXFP4 12.7 -> 11.4 us.
__device__ __forceinline__ void products8(const u32x4& a, const u32x4& b, float (&p)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t x = a[j], y = b[j];
    asm("v_fma_mix_f32 %0, %1, %2, neg(0) op_sel_hi:[1,1,0]" : "=v"(p[2 * j]) : "v"(x), "v"(y));
    asm("v_fma_mix_f32 %0, %1, %2, neg(0) op_sel:[1,1,0] op_sel_hi:[1,1,0]" : "=v"(p[2 * j + 1]) : "v"(x), "v"(y));
  }
}

// 1 / sqrt(x): the hardware's estimate e0 (relative error d, 2^-26 or so) and one step of third order,
// y = e0 (1 + d + 3/2 d^2 ...) with 2 d = 1 - x e0^2; NaN for an infinite x.
__device__ __forceinline__ double inverse_root(double x) {
  const double y = __builtin_amdgcn_rsq(x);
  const double e = fma(-(x * y), y, 1.0);
  return fma(y * e, fma(e, 0.375, 0.5), y);
}

// WPR waves a row (1: four rows a block); NCH 8-column chunks a thread in registers, as they lie in
// memory (0: the row is read twice).  Times below and the launch's choice: device time with inputs that
// change from call to call.
template <bool BF16, bool W32, int OUT, int WPR, int NCH>
__global__ __launch_bounds__(WPR == 1 ? 256 : 64 * WPR) void k_rmsnorm(NormArgs a) {
  __shared__ double red[2][WPR];
  constexpr int kThreads = 64 * WPR;
  const int tid = WPR == 1 ? threadIdx.x & 63 : threadIdx.x;
  // Blocks go to the 8 XCDs in turn; renumbered so that 8 neighbouring rows, whose scale words share
  // lines, are written through one XCD's L2 (16384 rows of 1024 25.7 -> 24.1 us; whole eighths of the
  // rows an XCD cost 16384 of 8192 5 us of 188).
  const unsigned n = (unsigned)(WPR == 1 ? (a.rows + 3) >> 2 : a.rows), b = block_number();
  if (b >= n) return;  // the whole block
  const unsigned at = (b | 63u) < n ? (b & ~63u) | ((b & 7u) << 3) | ((b >> 3) & 7u) : b;
  const int64_t row = WPR == 1 ? (int64_t)at * 4 + (threadIdx.x >> 6) : (int64_t)at;
  if (row >= a.rows) return;  // the whole wave
  const int K = a.cols;
  // 8-column chunks: whole 16-byte groups of codes, whole words of scales
  const int nch = OUT == kNormMxfp4 ? (K + 127) / 128 * 16 : OUT == kNormInt8 ? (K + 15) / 16 * 2 : (K + 7) / 8;
  const uint16_t* x = a.x + row * a.ldx;
  const uint16_t* r = a.r ? a.r + row * a.ldr : nullptr;
  uint16_t* hrow = a.r ? a.h + row * a.ldh : nullptr;

  double sum = 0.0, top = 0.0;
  // the sum of x and r, stored
  auto take = [&](int ch, const u32x4& xv, const u32x4& rv) {
    if (!r) return xv;
    float h[8], t[8];
    values8<BF16>(xv, h);
    values8<BF16>(rv, t);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = h[j] + t[j];
    const u32x4 p = pack8<BF16>(h);
    store8(hrow, 8 * ch, K, p);  // (stored past the caches, large sums cost the same, 16384 x 8192 2 % more)
    return p;
  };
  auto add = [&](const u32x4& p, const Weights<BF16, W32>& wv) {
    float h[8];
    values8<BF16>(p, h);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fma((double)h[j], (double)h[j], sum);
    if constexpr (OUT == kNormInt8) {
      float w[8];
      if constexpr (!BF16 && !W32) products8(p, wv.r[0], w);
      else wv.values(w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double v = !BF16 && !W32 ? (double)w[j] : (double)h[j] * (double)w[j];
        top = fmax(top, fabs(v));
        sum = fma(v, 0.0, sum);  // an infinite or NaN weight makes the row NaN
      }
    }
  };
  u32x4 h[NCH > 0 ? NCH : 1];
  Weights<BF16, W32> w[NCH > 0 ? NCH : 1];
  if constexpr (NCH > 0) {
    // all loads before the first store (h may be x or r themselves)
    u32x4 rv[NCH];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int ch = tid + c * kThreads;
      if (ch < nch) {
        h[c] = raw8(x, 8 * ch, K);
        if (r) rv[c] = raw8(r, 8 * ch, K);
        if constexpr (OUT == kNormInt8) w[c].load(a.w, 8 * ch, K);
      }
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int ch = tid + c * kThreads;
      if (ch < nch) {
        h[c] = take(ch, h[c], rv[c]);
        add(h[c], w[c]);
      }
    }
  } else {
    for (int ch = tid; ch < nch; ch += kThreads) {
      const u32x4 xv = raw8(x, 8 * ch, K);
      if constexpr (OUT == kNormInt8) w[0].load(a.w, 8 * ch, K);
      add(take(ch, xv, r ? raw8(r, 8 * ch, K) : xv), w[0]);
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
  // what is kept of the row stays as it lies in memory: without this its conversions are kept instead
  if constexpr (NCH > 0) {
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      asm volatile("" : "+v"(h[c]));
      if constexpr (OUT == kNormInt8) asm volatile("" : "+v"(w[c].r[0]));
      if constexpr (OUT == kNormInt8 && W32) asm volatile("" : "+v"(w[c].r[1]));
    }
  }

  RowStep st;
  if constexpr (OUT == kNormInt8) {
    // top is at least 0 and inv positive, or inv is NaN
    st = row_step(__builtin_bit_cast(uint32_t, (float)(top * inv)) & 0x7fffffffu);
    if (tid == 0) ((float*)a.scales)[row] = st.step;
  }
  auto write = [&](int ch, const u32x4& p, const Weights<BF16, W32>& wp) {
    float v[8];
    if constexpr (!BF16 && !W32) {
      products8(p, wp.r[0], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (float)((double)v[j] * inv);
    } else {
      float hc[8], wv[8];
      values8<BF16>(p, hc);
      wp.values(wv);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = (float)((double)hc[j] * (double)wv[j] * inv);
    }
    if constexpr (OUT == kNormSame) {
      store8((uint16_t*)a.y + row * a.ldy, 8 * ch, K, pack8<BF16>(v));
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
      if (ch < nch) {
        // (kept in registers from the start they cost more waves than their wait does time: 16384 rows of
        // 8192 189 us, loaded here 174)
        if constexpr (OUT != kNormInt8) w[c].load(a.w, 8 * ch, K);
        write(ch, h[c], w[c]);
      }
    }
  } else {
    for (int ch = tid; ch < nch; ch += kThreads) {
      w[0].load(a.w, 8 * ch, K);
      write(ch, raw8(r ? hrow : x, 8 * ch, K), w[0]);
    }
  }
}

template <bool BF16, bool W32, int OUT>
hipError_t launch_out(const NormArgs& a, hipStream_t stream) {
  const int nch = (a.cols + 127) / 128 * 16;
#define AWQ_NORM(W, N)                                                                           \
  hipLaunchKernelGGL((k_rmsnorm<BF16, W32, OUT, W, N>), grid_of(W == 1 ? (a.rows + 3) / 4 : a.rows), \
                     dim3(W == 1 ? 256 : 64 * W), 0, stream, a)
  // Waves a row, in us, with a residual and an fp32 weight: few rows wait for their loads (1 of 8192 to MXFP4:
  // two waves 8.0, four 5.3, eight 4.0; 256 of 5120 7.0, 5.7, 5.0; 500 of 16000 four 16.7, eight 14.8), many want
  // theirs close to full waves without a barrier among many (16384 of 256 to MXFP4: one wave 11.8, two 15.1, four
  // 20.5; of 1024 24.3, 24.4, 28.7; 4096 of 4096 to 8 bits 65, 28.7, 25.1, eight 27.7).
  if (a.rows > 1024 && nch <= 64) AWQ_NORM(1, 1);
  else if (a.rows > 1024 && nch <= 128) AWQ_NORM(2, 1);
  else if (a.rows > 1024 && nch <= 256) AWQ_NORM(4, 1);
  else if (a.rows > 1024 && nch <= 2 * 256) AWQ_NORM(4, 2);
  else if (a.rows > 1024 && nch <= 3 * 256) AWQ_NORM(4, 3);
  else if (a.rows > 1024 && nch <= 4 * 256) AWQ_NORM(4, 4);
  else if (nch <= 512) AWQ_NORM(8, 1);
  else if (nch <= 2 * 512) AWQ_NORM(8, 2);
  else if (nch <= 4 * 512) AWQ_NORM(8, 4);
  else AWQ_NORM(8, 0);
#undef AWQ_NORM
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t stream) {
  if (a.rows <= 0) return hipSuccess;
#define AWQ_NORM_OUT(B, W)                                             \
  a.out == kNormSame   ? launch_out<B, W, kNormSame>(a, stream)        \
  : a.out == kNormInt8 ? launch_out<B, W, kNormInt8>(a, stream)        \
                       : launch_out<B, W, kNormMxfp4>(a, stream)
  const bool w32 = a.w && a.w32;
  if (a.bf16) return w32 ? (AWQ_NORM_OUT(true, true)) : (AWQ_NORM_OUT(true, false));
  return w32 ? (AWQ_NORM_OUT(false, true)) : (AWQ_NORM_OUT(false, false));
#undef AWQ_NORM_OUT
}

}  // namespace awq
