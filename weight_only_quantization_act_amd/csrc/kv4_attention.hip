// Attention over the 4-bit key/value cache.
//
//   s_t = scale q . k_t,  k_t = step_t (c_t - z_t)  =>  s_t = scale step_t (q . c_t - z_t sum q)
//   out = sum_t e^{s_t} v_t / sum_t e^{s_t},  v_t = step'_t (c'_t - z'_t)
//       = (sum_t w_t c'_t - sum_t w_t z'_t) / sum_t e^{s_t},  w_t = e^{s_t} step'_t
// (per group of channels for the steps and zeros).  So the matrix cores multiply the raw codes,
// and step and zero enter once per score instead of once per channel.
//
// Pages: kwkr.cn AWQ 技术解析 §1.2, §4.2 (dequantisation fused into the product), lnrq.cn §四
// (decoding is bound by reading what was quantised).
//
// Codes as operands: a nibble in the top four mantissa bits of a fp16 pattern whose other bits
// are those of 16.0 is the number 16 + c, exactly: a shift and a v_and_or per pair of codes.
// The 16 goes into the zeros' sums: fp32 rounds at sum w (c + z + 32), which a key of a large step
// raises even where its code is its zero.  (Lower bits would save shifts and cost accuracy: 64 + c or
// 1024 + c cancel more of the fp32 sums, and the subnormals c 2^-24 lose their leading zeros in
// the matrix cores, which align the terms of a sum by their exponent fields: 2^-17 of the sum,
// measured.)  The cache's word order (awq_serve.h) is the operand order of these instructions.
//
// One wave, one tile of 32 keys, 16 columns (query rows x heads of the key head):
//   S = K Q^T   two 16 x 16 results; result row 4 q + e of result j is key 8 q + 4 j + e, so that
//               lane (column h, q) ends with the scores of keys 8 q .. 8 q + 7 of its column,
//               which is the layout of an operand of the next product: no data moves between
//               lanes.
//   O = V^T W   D / 16 results, row 4 q + e of result n is channel 16 n + 4 q + e.
// The reference of the exponents is per column and follows the running maximum with a slack of
// 2^kSlack, so that after the first tiles hardly any tile has to rescale what was summed
// (without it a column of random scores does so in one of t tiles after t, the wave's 16 or 32
// columns in nearly all of the first few dozen).  The weights are scaled by 2^f, f so chosen
// from the largest finite value step that the column has seen that w 2^f stays below 2^15: fp16
// holds them with full precision down to 2^-29 of the largest (a step of a masked key, NaN or
// infinite, does not count, or it would cost the others their precision).  A rise of the maximum or
// of that step multiplies what was summed so far by exp2 of the difference.  The weights' 11 bits are a
// choice: the error against 64 bits is 0.00022 to 0.00027 of an fp16 output's norm where fp32 weights
// leave the output's own rounding, 0.00020 (bf16: 0.0017 both); a second fp16 part of each weight would double
// the second product's instructions.
//
// Two forms.  Up to 16 columns (decode): a block's waves share the columns and take the tiles in
// turn, each with a ring of tiles in LDS that DMAs fill ahead; bound by the reading of the codes
// and by the vector instructions that make operands of them (two a pair of codes, about 350 a
// tile).  64 sequences of 2000 to 8192 tokens, 64 heads on 8 key heads of 128, groups of 64:
// 91 us, 4.1 TB/s of codes and parameters; one of 131072 tokens, groups of 128: 38 us, 3.7 TB/s.
// More columns (prompts): column tiles a wave, and the codes are decoded once a block; registers and
// LDS leave two waves a SIMD, which fill neither the vector unit (55% of the cycles: softmax, decoding)
// nor the matrix cores (28%).  A prompt of 4096 tokens, 32 heads on 8: 188 us, 0.73 PFLOP/s.  One
// form for both would decode the codes once a column tile (the prompt: 523 us), or leave three of four waves without work at a single token.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "grid.h"
#include "int8_quant.h"
#include "kv4_cache.h"
#include "mfma_dma.h"

namespace awq {

namespace {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8v __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

constexpr float kSlack = 4.0f;
constexpr float kNegInf = -__builtin_inff();
constexpr int kWaves = 4;
constexpr int kStages = 3;  // tiles a wave has in flight

__device__ __forceinline__ float max_q(float v) {  // over the four lanes of a column
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float sum_q(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// The operand pairs of one word: nibbles (n, n + 4) for n = 0..3, each as 16 + c.
constexpr uint32_t kNibble = 0x03C003C0u, kOffset = 0x4C004C00u;
constexpr float kOffsetF = 16.0f;
// The two constants in registers, the mask in a scalar and the offset in a vector one: a
// three-operand instruction takes one scalar and no literal, and with a literal each the
// compiler splits v_and_or_b32 in two.
struct CodeConsts {
  uint32_t mask, offset;
};
__device__ __forceinline__ CodeConsts code_consts() {
  CodeConsts c;
  asm volatile("s_mov_b32 %0, %1" : "=s"(c.mask) : "i"(kNibble));
  asm volatile("v_mov_b32 %0, %1" : "=v"(c.offset) : "i"(kOffset));
  return c;
}
template <int N>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, const CodeConsts& cc) {
  constexpr int S = 6 - 4 * N;
  return ((S > 0 ? w << (S > 0 ? S : 0) : w >> (S > 0 ? 0 : -S)) & cc.mask) | cc.offset;
}
__device__ __forceinline__ half8v word_operand(uint32_t w, const CodeConsts& cc) {
  const u32x4 v = {code_pair<0>(w, cc), code_pair<1>(w, cc), code_pair<2>(w, cc), code_pair<3>(w, cc)};
  return __builtin_bit_cast(half8v, v);
}

// exponent e with 2^e <= v < 2^(e+1), for a positive normal v; -127 for a subnormal
__device__ __forceinline__ int exponent_of(float v) {
  return (int)(__builtin_bit_cast(uint32_t, v) >> 23 & 255u) - 127;
}

template <int D, int GS>
struct Geo {
  static constexpr int G = D / GS;          // groups
  static constexpr int KW = D / 32;         // code words of a key and lane
  static constexpr int WPG = GS / 32;       // of them, words a group
  static constexpr int H = D / 64;          // 16-byte pieces of a lane's values of 8 tokens
  static constexpr int N = D / 16;          // value results
};

// Codes and parameters of one tile, one lane's part.
template <int D, int GS>
struct TileRegs {
  using X = Geo<D, GS>;
  uint32_t k[2][X::KW];
  u32x4 v[X::H];
  u32x4 kp[X::G][2], vp[X::G][2];
};

// A stage of a wave's ring in LDS: one tile, [K pieces][V pieces][G][K params | V params].  It is
// filled by DMA (no registers wait for data in flight) in the order in which the lanes read it
// back: the 16-byte pieces of K and V by lane, a group's parameters by key.
template <int D, int GS>
struct Ring {
  using X = Geo<D, GS>;
  static constexpr int KB = 16 * D, VB = 16 * D, BYTES = KB + VB + 256 * X::G;
  static constexpr int DMAS = KB / 1024 + VB / 1024 + X::G;  // a stage, a wave
};

// lane l's 16 (4) bytes at its address land at LDS byte lds + 16 l (4 l); see mfma_dma.h.
__device__ __forceinline__ void dma_piece(unsigned lds, const uint8_t* p) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               : : "s"(lds), "v"(p) : "memory", "m0");
}
__device__ __forceinline__ void dma_word(unsigned lds, const uint8_t* p) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
               : : "s"(lds), "v"(p) : "memory", "m0");
}
template <int N>
__device__ __forceinline__ void wait_dma() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "i"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); }

// Byte offsets of a lane's pieces from a tile's first key (K, V) and of its parameter words.
template <int D, int GS>
struct LaneOffsets {
  int k[Ring<D, GS>::KB / 1024], v, par;  // V pieces are 256 bytes apart, groups 4 P
  int k_half, v_half, par_half;           // which 16 keys of the tile they belong to
};
template <int D, int GS>
__device__ __forceinline__ LaneOffsets<D, GS> lane_offsets(int lane, int P) {
  using X = Geo<D, GS>;
  LaneOffsets<D, GS> o;
  const int lr = lane & 15, q = lane >> 4;
  const int key = 8 * (lr >> 2) + (lr & 3);  // + 4 j: the key of result row lr of result j
  if constexpr (D == 128) {
    o.k[0] = key * 64 + q * 16;
    o.k[1] = o.k[0] + 4 * 64;
  } else {  // a piece holds the words of two lanes: [j][piece of the row][row]
    o.k[0] = (key + 4 * (lane >> 5)) * 32 + (q & 1) * 16;
  }
  o.k_half = lr >> 3;
  o.v = q * 4 * D + lr * 16;
  o.v_half = q >> 1;
  o.par = (lane & 31) * 4 + (lane >> 5) * 4 * P * X::G;
  o.par_half = (lane >> 4) & 1;
  return o;
}

// Start the DMAs of one tile: keys [off, off + 32) of the page at ra if it holds them all, else
// (pages of 16) the pages at ra and rb.
template <int D, int GS>
__device__ __forceinline__ void dma_tile(unsigned lds, const uint8_t* ra, const uint8_t* rb, int off,
                                         int P, const LaneOffsets<D, GS>& o) {
  using X = Geo<D, GS>;
  using R = Ring<D, GS>;
  const uint8_t* k = ra + off * (D / 2);
  const uint8_t* v = ra + P * (D / 2) + off * (D / 2);
  const uint8_t* p = ra + P * D + 4 * off;
  if (P == 16) {  // the second half's addresses count from the tile's first key too
    k = o.k_half ? rb - 16 * (D / 2) : k;
    v = o.v_half ? rb + P * (D / 2) - 16 * (D / 2) : v;
    p = o.par_half ? rb + P * D - 64 : p;
  }
#pragma unroll
  for (int i = 0; i < R::KB / 1024; ++i) dma_piece(lds + 1024 * i, k + o.k[i]);
#pragma unroll
  for (int h = 0; h < X::H; ++h) dma_piece(lds + R::KB + 1024 * h, v + o.v + 256 * h);
#pragma unroll
  for (int g = 0; g < X::G; ++g) dma_word(lds + R::KB + R::VB + 256 * g, p + o.par + 4 * P * g);
}

template <int D, int GS>
__device__ __forceinline__ void read_tile(TileRegs<D, GS>& r, const uint8_t* st, int lane) {
  using X = Geo<D, GS>;
  using R = Ring<D, GS>;
  const int q = lane >> 4;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if constexpr (D == 128) {
      const u32x4 w = *(const u32x4*)(st + 1024 * j + 16 * lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) r.k[j][e] = w[e];
    } else {
      const uint2 w = *(const uint2*)(st + 512 * j + (q >> 1) * 256 + (lane & 15) * 16 + (q & 1) * 8);
      r.k[j][0] = w.x;
      r.k[j][1] = w.y;
    }
  }
#pragma unroll
  for (int h = 0; h < X::H; ++h) r.v[h] = *(const u32x4*)(st + R::KB + 1024 * h + 16 * lane);
  const uint8_t* par = st + R::KB + R::VB + 32 * q;
#pragma unroll
  for (int g = 0; g < X::G; ++g)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      r.kp[g][i] = *(const u32x4*)(par + 256 * g + 16 * i);
      r.vp[g][i] = *(const u32x4*)(par + 256 * g + 128 + 16 * i);
    }
}

// A column tile's state in one wave.
template <int D, int GS>
struct Column {
  using X = Geo<D, GS>;
  half8v q[X::KW];     // operands of S, in word order
  f32x4 c16[X::G];     // -16 times the sum of a group's q: what S starts from
  float qsum[X::G];    // sum of a group's q
  float sigma;         // from the raw score to log2 units
  int pos;             // the row's position; -1: no row
  float m;             // reference of the scores, log2 units: their maximum to within kSlack
  uint32_t limit;      // fp16 pattern that the value steps seen lie below; 0 before the first tile
  float nM;            // f - m: weights are exp2(s + nM); 0 before the first key
  float l;             // this lane's sum of exp2(s + nM)
  f32x4 z[X::G];       // sum of weight x (zero + 16): every row the same
  f32x4 o[X::N];
  __device__ float M() const { return m == kNegInf ? kNegInf : -nM; }
};

// The lane's part of one row of q, in word order (zeros without a row).
template <int D, int GS>
struct QueryRow {
  uint4 w[Geo<D, GS>::KW];
};
template <int D, int GS>
__device__ __forceinline__ QueryRow<D, GS> read_query(const uint16_t* row, int q) {
  using X = Geo<D, GS>;
  QueryRow<D, GS> r;
#pragma unroll
  for (int w = 0; w < X::KW; ++w) {
    r.w[w] = uint4{0u, 0u, 0u, 0u};
    if (row) r.w[w] = *(const uint4*)(row + (w / X::WPG) * GS + q * (GS / 4) + (w % X::WPG) * 8);
  }
  return r;
}

// A row of q as operands: scaled by a power of two so that its largest magnitude lies in
// [2^8, 2^9), then rounded to fp16 (exact but for what lies 2^-24 and more below the largest).
template <int D, int GS>
__device__ __forceinline__ void set_query(Column<D, GS>& c, const QueryRow<D, GS>& row, bool bf16,
                                          float scale) {
  using X = Geo<D, GS>;
  float v[X::KW][8];
  float top = 0.0f;
#pragma unroll
  for (int w = 0; w < X::KW; ++w) {
    const uint32_t r[4] = {row.w[w].x, row.w[w].y, row.w[w].z, row.w[w].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[w][2 * i] = bf16 ? from16<true>(r[i] & 0xffffu) : from16<false>(r[i] & 0xffffu);
      v[w][2 * i + 1] = bf16 ? from16<true>(r[i] >> 16) : from16<false>(r[i] >> 16);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[w][i]));
  }
  top = max_q(top);
  // an infinity makes the row NaN here already: a sum of products that happened to be -infinity for every
  // key would pass for a row without keys
  const float poison = top < __builtin_inff() ? 0.0f : __builtin_nanf("");
  // -119 .. 135 (a subnormal counts as 2^-127); a row of zeros is left as it is
  const int e = top > 0.0f && top < __builtin_inff() ? 8 - exponent_of(top) : 0;
  // scale log2(e) 2^-e, in the order in which nothing on the way leaves fp32's range
  constexpr float kLog2e = 1.44269504088896340736f;
  c.sigma = e < 0 ? ldexpf(scale, -e) * kLog2e : ldexpf(scale * (0.5f * kLog2e), 1 - e);
  // a factor of 0 or infinity would make NaN of masked scores, -infinity, or of scores of 0.  Raw scores
  // stay below 2^38, so that under the least normal factor each weight is 1; where the largest is short
  // of scale log2(e) 2^-e, scores other than 0 decide alone or leave fp32's range
  c.sigma = fminf(fmaxf(c.sigma, 0x1p-126f), 0x1.fffffep127f);
#pragma unroll
  for (int g = 0; g < X::G; ++g) c.qsum[g] = 0.0f;
#pragma unroll
  for (int w = 0; w < X::KW; ++w) {
    half8v h;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const _Float16 lo = (_Float16)(ldexpf(v[w][n], e) + poison),
                     hi = (_Float16)(ldexpf(v[w][n + 4], e) + poison);
      h[2 * n] = lo;
      h[2 * n + 1] = hi;
      c.qsum[w / X::WPG] += (float)lo + (float)hi;
    }
    c.q[w] = h;
  }
#pragma unroll
  for (int g = 0; g < X::G; ++g) {
    c.qsum[g] = sum_q(c.qsum[g]);
    const float x = -kOffsetF * c.qsum[g];
    c.c16[g] = f32x4{x, x, x, x};
    c.z[g] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  c.m = kNegInf;
  c.limit = 0;
  c.nM = 0.0f;
  c.l = 0.0f;
#pragma unroll
  for (int n = 0; n < X::N; ++n) c.o[n] = f32x4{0.f, 0.f, 0.f, 0.f};
}

// Two floats as a pair of fp16, nearest even.
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pair16(float x, float y) {
  const f32x2 v = {x, y};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, half2v));
}

__device__ __forceinline__ float lo16(uint32_t w) { return h2f((uint16_t)w); }
__device__ __forceinline__ float hi16(uint32_t w) { return h2f((uint16_t)(w >> 16)); }

// The power of two f of a column's weights: w = exp2(s - m + f) step stays below 2^15 for steps below
// the fp16 pattern `limit`, a whole exponent, 1 << 10 and more.
__device__ __forceinline__ float weight_exponent(uint32_t limit) {
  return 14.0f - kSlack + 15.0f + 1.0f - (float)(limit >> 10);
}
// `limit` raised above the pattern of a step (zero and subnormal steps count as the smallest normal
// one).
__device__ __forceinline__ uint32_t limit_above(uint32_t step, uint32_t limit) {
  return max(limit, ((max(step, 0x0400u) >> 10) + 1) << 10);
}
// The step of a parameter word if it counts: its key is seen and it is finite.
__device__ __forceinline__ uint32_t counted_step(uint32_t par, bool seen) {
  const uint32_t s = par & 0xffffu;
  return seen && s < 0x7c00u ? s : 0u;
}
// The halves of a pair of keys that are seen (bits e and e + 1).
__device__ __forceinline__ uint32_t seen_halves(uint32_t seen, int e) {
  return (seen >> e & 1 ? 0xffffu : 0u) | (seen >> (e + 1) & 1 ? 0xffff0000u : 0u);
}
// The steps of a pair of parameter words.
__device__ __forceinline__ uint32_t step_pair(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x05040100u);
}

// One tile of 32 keys.  !whole (the same in every lane): some (key, column) pairs do not exist;
// key0 is the tile's first key, lo_off = window - 1 (or a huge number) so that column pos sees keys
// [pos - lo_off, pos]; dead: bit x set if the keys of half x lie on no page.
template <int D, int GS>
__device__ __forceinline__ void do_tile(TileRegs<D, GS>& r, Column<D, GS>& c, bool whole,
                                        int key0, int n_keys, int lo_off, int dead,
                                        const CodeConsts& cc, int lane) {
  using X = Geo<D, GS>;
  const int q = lane >> 4;
  const int kq = key0 + 8 * q;
  int there = 8;  // keys kq .. kq + there - 1 exist
  if (!whole) {
    there = (dead >> (q >> 1)) & 1 ? 0 : n_keys - kq;
    asm volatile("" : "+v"(there));  // (keeps the comparisons inside these branches)
    // parameters of keys that do not exist may hold anything
#pragma unroll
    for (int g = 0; g < X::G; ++g)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        r.kp[g][e >> 2][e & 3] = e < there ? r.kp[g][e >> 2][e & 3] : 0u;
        r.vp[g][e >> 2][e & 3] = e < there ? r.vp[g][e >> 2][e & 3] : 0u;
      }
  }
  // largest value step of the lane's keys (as fp16 patterns; the packed maximum also forms that
  // of the zeros, unused)
  u16x2 tp = {0, 0};
#pragma unroll
  for (int g = 0; g < X::G; ++g)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t w = r.vp[g][e >> 2][e & 3];
      tp = __builtin_elementwise_max(tp, __builtin_bit_cast(u16x2, w));
    }
  const uint32_t top = tp[0];

  float s[8];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
#pragma unroll
    for (int g = 0; g < X::G; ++g) {
      f32x4 a = c.c16[g];
#pragma unroll
      for (int u = 0; u < X::WPG; ++u)
        a = __builtin_amdgcn_mfma_f32_16x16x32_f16(word_operand(r.k[j][g * X::WPG + u], cc),
                                                   c.q[g * X::WPG + u], a, 0, 0, 0);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t w = r.kp[g][j][e];
        const float x = fmaf(-hi16(w), c.qsum[g], a[e]);
        s[4 * j + e] = fmaf(lo16(w), x, g == 0 ? 0.0f : s[4 * j + e]);
      }
    }
  }
  float mn = s[0];  // the least score of a key that is seen
#pragma unroll
  for (int e = 1; e < 8; ++e) mn = fminf(mn, s[e]);
  uint32_t seen = 0xff;  // bit e: key 8 q + e exists for the column
  if (!whole) {
    seen = 0;
    int last = min(there - 1, c.pos - kq), fst = c.pos - lo_off - kq;
    asm volatile("" : "+v"(last), "+v"(fst));
    mn = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool ok = e <= last && e >= fst;
      mn = ok ? fminf(mn, s[e]) : mn;
      s[e] = ok ? s[e] : kNegInf;
      seen |= ok ? 1u << e : 0u;
    }
  }
  float mx = s[0];
#pragma unroll
  for (int e = 1; e < 8; ++e) mx = fmaxf(mx, s[e]);
  // a key of infinite step is NaN, also where what it gives is -infinity, as if it were not there
  if (mn == kNegInf) c.l = __builtin_nanf("");
  mx *= c.sigma;
  // seldom: a score above the column's maximum, or a value step above what the weights' scale
  // was made for
  if (__any(mx > c.m + kSlack || top >= c.limit)) {
    uint32_t all = top;
    if (!whole) {  // of keys that the column sees
      tp = u16x2{0, 0};
#pragma unroll
      for (int g = 0; g < X::G; ++g)
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const u32x4 w = r.vp[g][e >> 2];
          tp = __builtin_elementwise_max(
              tp, __builtin_bit_cast(u16x2, step_pair(w[e & 3], w[(e & 3) + 1]) & seen_halves(seen, e)));
        }
      all = max(tp[0], tp[1]);
    }
    if (__any(all >= 0x7c00u)) {  // NaN or infinite: the largest of the others
      all = 0;
#pragma unroll
      for (int g = 0; g < X::G; ++g)
#pragma unroll
        for (int e = 0; e < 8; ++e) all = max(all, counted_step(r.vp[g][e >> 2][e & 3], seen >> e & 1));
    }
    all = max(all, (uint32_t)__shfl_xor((int)all, 16));
    all = max(all, (uint32_t)__shfl_xor((int)all, 32));
    c.limit = limit_above(all, c.limit);
    const float m = fmaxf(c.m, max_q(mx));
    const float nM = m == kNegInf ? 0.0f : weight_exponent(c.limit) - m;
    const float a = c.m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(nM - c.nM);
    c.m = m;
    c.nM = nM;
    c.l *= a;
#pragma unroll
    for (int g = 0; g < X::G; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) c.z[g][e] *= a;
#pragma unroll
    for (int n = 0; n < X::N; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) c.o[n][e] *= a;
  }
  float p[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    p[e] = __builtin_amdgcn_exp2f(fmaf(s[e], c.sigma, c.nM));
    c.l += p[e];
  }
#pragma unroll
  for (int g = 0; g < X::G; ++g) {
    u32x4 w, zo;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t pa = r.vp[g][i >> 1][2 * (i & 1)], pb = r.vp[g][i >> 1][2 * (i & 1) + 1];
      w[i] = pair16(fmaf(p[2 * i], lo16(pa), 0.0f), fmaf(p[2 * i + 1], lo16(pb), 0.0f));
      // zeros + 16, exact in fp16
      zo[i] = __builtin_bit_cast(
          uint32_t, __builtin_bit_cast(half2v, __builtin_amdgcn_perm(pb, pa, 0x07060302u)) +
                        __builtin_bit_cast(half2v, kOffset));
    }
    if (!whole) {  // a masked key's step may be NaN
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] &= (seen >> (2 * i) & 1 ? 0xffffu : 0u) | (seen >> (2 * i + 1) & 1 ? 0xffff0000u : 0u);
    }
    // the zeros' sum by the same instruction as the codes' (an operand whose 16 rows are
    // equal), so that what the two sums share cancels as it was rounded
    c.z[g] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8v, zo),
                                                    __builtin_bit_cast(half8v, w), c.z[g], 0, 0, 0);
#pragma unroll
    for (int n = g * (GS / 16); n < (g + 1) * (GS / 16); ++n) {
      const u32x4 vw = r.v[n >> 2];
      u32x4 a;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        a[i] = (n & 3) == 0   ? code_pair<0>(vw[i], cc)
               : (n & 3) == 1 ? code_pair<1>(vw[i], cc)
               : (n & 3) == 2 ? code_pair<2>(vw[i], cc)
                              : code_pair<3>(vw[i], cc);
      c.o[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8v, a),
                                                     __builtin_bit_cast(half8v, w), c.o[n], 0, 0, 0);
    }
  }
}

// Results of a column tile: sums over the column's lanes, the zeros subtracted.  o is then
// sum_t w_t (c - z), l the weights' sum, both over exp2(M()).
template <int D, int GS>
__device__ __forceinline__ void finish(Column<D, GS>& c) {
  using X = Geo<D, GS>;
  c.l = sum_q(c.l);
#pragma unroll
  for (int g = 0; g < X::G; ++g) {
#pragma unroll
    for (int n = g * (GS / 16); n < (g + 1) * (GS / 16); ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) c.o[n][e] -= c.z[g][e];
  }
}

__device__ __forceinline__ void store4(void* out, int64_t at, bool bf16, const float (&v)[4]) {
  uint2 w;
  if (bf16) {
    w.x = to16<true>(v[0]) | ((uint32_t)to16<true>(v[1]) << 16);
    w.y = to16<true>(v[2]) | ((uint32_t)to16<true>(v[3]) << 16);
  } else {
    w.x = to16<false>(v[0]) | ((uint32_t)to16<false>(v[1]) << 16);
    w.y = to16<false>(v[2]) | ((uint32_t)to16<false>(v[3]) << 16);
  }
  *(uint2*)((uint16_t*)out + at) = w;
}

__device__ __forceinline__ float lse_of(float M, float l) {
  return l == 0.0f ? kNegInf : (M + __builtin_amdgcn_logf(l)) * 0.69314718055994530942f;
}

// Workspace of a call whose keys are divided, fp32: o [slot][D], then (M, l) [slot].
//   wide: slot = (token, head) x splits.
//   decode: slot = (key head, place) x 16 columns; then int32 [sequence][key head] x 2: the first
//   place of a sequence's parts and their number.
struct Partials {
  float* o;
  float* ml;
  int32_t* parts;
  int splits, tiles;
};

// Which work a block of the wide form does.  Blocks start in the order of their number: later
// column tiles see more keys, so they go first, of all heads before any earlier tile (a prompt of 4096
// tokens: 302 us with a head's tiles together, when long blocks start late, 211 so).  Consecutive
// blocks, which go to different dies, are different key heads: with eight of them each die's L2
// holds one.  Sequences follow one another, so that it holds one sequence of that head (four
// prompts of up to 8192 tokens: 2430 us with the sequences' tiles in turn, 1413 so).
struct Place {
  int head, split, seq, tile;  // tile -1: none
};
__device__ __forceinline__ Place place_of(const Kv4Cache& c, const Partials& part) {
  unsigned n = block_number();
  Place p;
  p.head = n % c.kv_heads;
  n /= c.kv_heads;
  p.split = n % part.splits;
  n /= part.splits;
  p.tile = part.tiles - 1 - (int)(n % part.tiles);
  p.seq = n / part.tiles;
  if (p.seq >= c.n_seqs) p.tile = -1;
  return p;
}

// A sequence of a call with few columns: its rows, its keys and the tiles that some row sees.
struct Extent {
  int row0, rows, len, pos0;  // first row, rows, keys that are there, position of the first row
  int t_lo, t_hi;             // tiles of 32 keys
  // what it counts in the division of the work: a sequence without keys still has rows to write
  __device__ unsigned weight() const { return rows > 0 ? (unsigned)max(1, t_hi - t_lo) : 0u; }
};
__device__ __forceinline__ Extent extent_of(const Kv4Cache& c, const Kv4Query& a, int b) {
  // (not written here: scalar loads where b is the same in all lanes)
  const auto* starts = (const __attribute__((address_space(4))) int32_t*)(uintptr_t)c.starts;
  const auto* lens = (const __attribute__((address_space(4))) int32_t*)(uintptr_t)c.lens;
  Extent e;
  e.row0 = starts[b];
  const int count = starts[b + 1] - e.row0, len0 = lens[b];
  e.rows = min(min(count, a.max_q), (int)a.n_tokens - e.row0);
  // bounded by the table and by the caller's bound
  e.len = min(len0, (int)min((int64_t)c.max_blocks << c.log2p, (int64_t)a.max_len));
  e.pos0 = len0 - count;
  const int lo_off = a.window > 0 ? a.window - 1 : 0x3fffffff;
  e.t_lo = max(0, e.pos0 - lo_off) >> 5;
  e.t_hi = max(e.t_lo, max(0, min(e.len, e.pos0 + e.rows) + 31) >> 5);
  return e;
}

__device__ __forceinline__ unsigned lane_value(unsigned v, int lane) {
  return (unsigned)__builtin_amdgcn_readlane((int)v, lane);
}

// sum over lanes 0 .. lane: within rows of 16 lanes, then their totals
__device__ __forceinline__ unsigned wave_scan(unsigned v) {
#define AWQ_SCAN(CTRL, ROWS) \
  v += (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false)
  AWQ_SCAN(0x111, 0xf);  // row_shr 1, 2, 4, 8
  AWQ_SCAN(0x112, 0xf);
  AWQ_SCAN(0x114, 0xf);
  AWQ_SCAN(0x118, 0xf);
  AWQ_SCAN(0x142, 0xa);  // lane 15 of a row to the next, rows 1 and 3
  AWQ_SCAN(0x143, 0xc);  // lane 31 to rows 2 and 3
#undef AWQ_SCAN
  return v;
}

// The division of the tiles of all sequences (of one key head) over `blocks` blocks: block j takes
// positions [j share, (j + 1) share) of the sequences' weights laid end to end (32 bits hold
// them: see kv4_plan).  Every wave works it out, 64 sequences at a time.
struct Share {
  unsigned total, share, at;  // at: the block's first position
  int seq;                    // the sequence there, -1: none
  unsigned offset;            // position within it
  Extent mine;                // of sequence base + lane
  int base;
};
__device__ __forceinline__ Share share_of(const Kv4Cache& c, const Kv4Query& a, int j, int blocks,
                                          int lane) {
  Share s;
  auto read = [&](int base) -> unsigned {
    s.base = base;
    s.mine = extent_of(c, a, min(base + lane, c.n_seqs - 1));
    return base + lane < c.n_seqs ? s.mine.weight() : 0u;
  };
  s.total = 0;
  unsigned v = 0, sum = 0;
  for (int base = 0; base < c.n_seqs; base += 64) {
    v = read(base);
    sum = wave_scan(v);
    s.total += lane_value(sum, 63);
  }
  s.share = max((s.total + blocks - 1) / blocks, 8u);
  s.at = s.share * j;
  s.seq = -1;
  s.offset = 0;
  if (s.at >= s.total) return s;
  unsigned before = 0;
  for (int base = 0; base < c.n_seqs; base += 64) {
    if (c.n_seqs > 64) {
      v = read(base);
      sum = wave_scan(v);
    }
    const unsigned all = lane_value(sum, 63);
    if (s.at < before + all) {
      const int who = __builtin_ctzll(__ballot(sum > s.at - before));
      s.seq = base + who;
      s.offset = s.at - before - (lane_value(sum, who) - lane_value(v, who));
      break;
    }
    before += all;
  }
  return s;
}
__device__ __forceinline__ Extent share_extent(const Share& s, const Kv4Cache& c, const Kv4Query& a, int b) {
  if (b - s.base >= 64) return extent_of(c, a, b);
  const int l = b - s.base;
  Extent e;
  e.row0 = (int)lane_value((unsigned)s.mine.row0, l);
  e.rows = (int)lane_value((unsigned)s.mine.rows, l);
  e.len = (int)lane_value((unsigned)s.mine.len, l);
  e.pos0 = (int)lane_value((unsigned)s.mine.pos0, l);
  e.t_lo = (int)lane_value((unsigned)s.mine.t_lo, l);
  e.t_hi = (int)lane_value((unsigned)s.mine.t_hi, l);
  return e;
}

// Waves a SIMD that the registers of the undivided form are kept to (divided, two blocks a compute
// unit are two waves a SIMD, and fewer registers would spill: one sequence of 131072 tokens, 44 us
// with three, 40 with two).
constexpr int waves_per_simd(int dim, int group) {
  return dim / group > 2 ? 2 : dim == 64 && group == 64 ? 4 : 3;
}

// Up to 16 columns (decode): the waves of a block share the columns and take the tiles in turn,
// a ring of kStages tiles each (64 sequences: 169 us with two stages, 96 with three, 97 with four).
// DIVIDED: the tiles of all sequences are dealt out evenly, so that a block may do parts of
// several sequences; a sequence that lies in one block is written from there, the parts of the
// others are joined by a second launch (64 sequences of 2000 to 8192 tokens: 96 us with a block a
// sequence and head, 101 with equal pieces of 2048 keys, 91 so).  Otherwise a block does one sequence.
template <int D, int GS, int WAVES, bool DIVIDED>
__global__ __launch_bounds__(64 * WAVES)
__attribute__((amdgpu_waves_per_eu(DIVIDED ? 2 : waves_per_simd(D, GS))))
void k_kv4_attention(Kv4Cache c, Kv4Query a, Partials part) {
  using X = Geo<D, GS>;
  using R = Ring<D, GS>;
  constexpr int NS = kStages, step = WAVES;
  constexpr int kRing = NS * R::BYTES * WAVES;
  constexpr int kJoin = WAVES * 16 * (D + 6) * (int)sizeof(float);
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kRing > kJoin ? kRing : kJoin];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const unsigned number = block_number();
  const int kvh = number % c.kv_heads, index = number / c.kv_heads;  // index: of the head's blocks
  const int group = a.heads / c.kv_heads;
  const int lo_off = a.window > 0 ? a.window - 1 : 0x3fffffff;
  const int P = 1 << c.log2p, n_pages = (int)c.n_pages;
  uint8_t* ring = lds + wave * (NS * R::BYTES);
  const unsigned ring_at = lds_address(ring);
  const LaneOffsets<D, GS> lo = lane_offsets<D, GS>(lane, P);
  const CodeConsts cc = code_consts();

  Share s;
  unsigned left;  // what the block still has to do
  if constexpr (DIVIDED) {
    s = share_of(c, a, index, part.splits, lane);
    if (s.seq < 0) return;  // the whole block
    left = min(s.share, s.total - s.at);
  } else {
    if (index >= c.n_seqs) return;
    s.seq = index;
    s.offset = 0;
    left = 1;
  }
  for (; left > 0; ++s.seq) {
    const int b = s.seq;
    const Extent ex = DIVIDED ? share_extent(s, c, a, b) : extent_of(c, a, b);
    const unsigned weight = ex.weight();
    if (weight == 0) {
      if (DIVIDED) continue;
      return;
    }
    const int len = ex.len, pos0 = ex.pos0, row0 = ex.row0, n_cols = ex.rows * group;
    const int last_i = ex.rows - 1;
    int t_lo = ex.t_lo, t_hi = ex.t_hi;
    bool whole_seq = true;
    if constexpr (DIVIDED) {
      const unsigned take = min(left, weight - s.offset);
      whole_seq = take == weight;
      t_lo += s.offset;
      t_hi = min(t_hi, t_lo + (int)take);
      if (s.offset == 0 && threadIdx.x == 0) {
        int2 w;
        w.x = index + b;
        w.y = (int)((s.at + weight - 1) / s.share) - index + 1;
        *(int2*)(part.parts + 2 * ((int64_t)b * c.kv_heads + kvh)) = w;
      }
      left -= take;
      s.at += take;
      s.offset = 0;
    } else {
      left = 0;
    }
    const int x = lane & 15, xi = x / group;
    const bool has = x < n_cols;
    const QueryRow<D, GS> query = read_query<D, GS>(
        has ? (const uint16_t*)a.q + (int64_t)(row0 + xi) * a.qt + (int64_t)(kvh * group + x - xi * group) * a.qh
            : nullptr,
        lane >> 4);
    // (the table is not written here: scalar loads)
    const auto* table = (const __attribute__((address_space(4))) int32_t*)(uintptr_t)(
        c.table + (int64_t)b * c.max_blocks);
    const int last_blk = max(0, (len - 1) >> c.log2p);
    const int t0 = t_lo + wave;
    // tiles t0, t0 + step, ...: tile i of the wave in stage i mod NS
    const int n_tiles = t_hi > t0 ? (t_hi - t0 + step - 1) / step : 0;
    int dead_of[NS];
    // the table entries of the next tile to start, read one tile ahead
    int page_a, page_b;
    auto look_up = [&](int i) {
      const int key = 32 * (t0 + i * step);
      page_a = table[min(key >> c.log2p, last_blk)];
      page_b = table[min((key + 16) >> c.log2p, last_blk)];
    };
    auto start = [&](int i, int s) {
      const int key = 32 * (t0 + i * step);
      const int bad_a = (unsigned)page_a >= (unsigned)n_pages, bad_b = (unsigned)page_b >= (unsigned)n_pages;
      const uint8_t* ra = c.pages + ((int64_t)(bad_a ? 0 : page_a) * c.kv_heads + kvh) * (int64_t)c.record;
      const uint8_t* rb = c.pages + ((int64_t)(bad_b ? 0 : page_b) * c.kv_heads + kvh) * (int64_t)c.record;
      look_up(i + 1);
      dead_of[s] = bad_a | (bad_b << 1);
      dma_tile<D, GS>(ring_at + s * R::BYTES, ra, rb, key & (P - 1), P, lo);
    };
    if (n_tiles > 0) look_up(0);
#pragma unroll
    for (int s = 0; s < NS; ++s)
      if (s < n_tiles) start(s, s);
    // the query's arithmetic while the first tiles come in
    Column<D, GS> col;
    set_query<D, GS>(col, query, a.bf16, a.scale);
    col.pos = has ? pos0 + xi : -1;
    for (int i0 = 0; i0 < n_tiles; i0 += NS) {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int i = i0 + s;
        if (i < n_tiles) {
          // this stage's DMAs have landed: NS - 1 later tiles may be in flight
          if (i + NS <= n_tiles) wait_dma<(NS - 1) * R::DMAS>();
          else wait_dma<0>();
          TileRegs<D, GS> r;
          read_tile<D, GS>(r, ring + s * R::BYTES, lane);
          wait_lds();  // the stage is in registers: refill it
          const int dead = dead_of[s];
          if (i + NS < n_tiles) start(i + NS, s);
          const int key0 = 32 * (t0 + i * step);
          // every key of the tile exists and every column sees all of it
          const bool whole = !dead && key0 + 32 <= len && key0 + 31 <= pos0 &&
                             key0 >= pos0 + last_i - lo_off;
          do_tile<D, GS>(r, col, whole, key0, len, lo_off, dead, cc, lane);
        }
      }
    }

    finish<D, GS>(col);

    {
      // the waves' results joined in wave order: each scaled to the block's largest M
      float (*so)[16][D + 4] = (float (*)[16][D + 4])lds;
      float (*sm)[16] = (float (*)[16])(so + WAVES);
      float (*sl)[16] = sm + WAVES;
      __syncthreads();  // the rings are done with
      const int cx = lane & 15;
#pragma unroll
      for (int n = 0; n < X::N; ++n) *(f32x4*)&so[wave][cx][16 * n + 4 * (lane >> 4)] = col.o[n];
      if ((lane >> 4) == 0) {
        sm[wave][cx] = col.M();
        sl[wave][cx] = col.l;
      }
      __syncthreads();
      // thread -> column, 4 channels at a time
      for (int w = threadIdx.x; w < 16 * (D / 4); w += 64 * WAVES) {
        const int cx = w / (D / 4), ch = (w % (D / 4)) * 4;
        if (cx >= n_cols) continue;
        float M = sm[0][cx];
#pragma unroll
        for (int i = 1; i < WAVES; ++i) M = fmaxf(M, sm[i][cx]);
        float l = 0.0f;
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < WAVES; ++i) {
          // a wave without a maximum has seen no key (sums 0) or only NaN (sums NaN, which stay)
          const float k = sm[i][cx] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(sm[i][cx] - M);
          l = fmaf(sl[i][cx], k, l);
          const f32x4 v = *(const f32x4*)&so[i][cx][ch];
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = fmaf(v[e], k, o[e]);
        }
        const int i = cx / group, h = cx - i * group;
        const int64_t r = (int64_t)(row0 + i) * a.heads + kvh * group + h;
        if (DIVIDED && !whole_seq) {
          const int64_t slot = ((int64_t)kvh * (part.splits + c.n_seqs) + index + b) * 16 + cx;
          *(f32x4*)(part.o + slot * D + ch) = o;
          if (ch == 0) *(float2*)(part.ml + slot * 2) = float2{M, l};
        } else {
          const float inv = l == 0.0f ? 0.0f : 1.0f / l;
          const float v[4] = {o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv};
          store4(a.out, r * D + ch, a.bf16, v);
          if (ch == 0 && a.lse) a.lse[r] = lse_of(M, l);
        }
      }
    }
    // the next sequence's tiles go where this one's sums lie
    if (DIVIDED && left > 0) __syncthreads();
  }
}

// ---- many columns (prompts) ---------------------------------------------------------------
//
// A block of four waves takes 16 NC columns a wave and walks the keys 64 at a time.  The codes
// are made operands once a block: each wave decodes a part of the next 64 keys, as the exact
// integers c - z in fp16, into LDS (two buffers, one barrier a step) while the codes after that
// are in flight to registers.  The steps stay fp32 factors of the scores and of the weights, as
// above, so a value is never rounded.
// (two do not fit the registers with four groups of 32 channels)
constexpr int wide_tiles(int dim, int group) { return dim / group > 2 ? 1 : 2; }

template <int D, int GS>
struct Wide {
  using X = Geo<D, GS>;
  static constexpr int NC = wide_tiles(D, GS);       // column tiles a wave
  static constexpr int COLS = 16 * NC * kWaves;      // columns a block
  static constexpr int K_BYTES = 2 * 2 * X::KW * 1024;  // [32 keys][result j][word][lane] pieces
  static constexpr int V_BYTES = 2 * X::N * 1024;       // [32 keys][value result][lane] pieces
  static constexpr int P_BYTES = 2 * X::G * 256;        // [K, V][group][64 keys] parameter words
  static constexpr int BYTES = K_BYTES + V_BYTES + P_BYTES;
};

// What a wave decodes of one step, in registers: the codes of a K pass (32 keys, result j) and
// of a V pass (32 keys, 16-byte piece h), the zeros they need, and its part of the parameters.
template <int D, int GS>
struct Raw {
  using X = Geo<D, GS>;
  static constexpr int GH = GS == 32 ? 2 : 1;        // groups of one V piece
  static constexpr int PW = (2 * X::G + kWaves - 1) / kWaves;  // parameter words a thread
  uint32_t k[X::KW], kz[X::G];
  u32x4 v, vz[GH][2];
  uint32_t par[PW];
  uint64_t dead;  // bit l: key l of the step lies on no page
  int v_there;    // of the 8 keys of v, those that exist
};

// Codes minus zeros, exact, without a shift per pair: a nibble in the low four bits of a half
// under the pattern of 1024 is 1024 + c, one in the next four under that of 64 is 64 + c, and
// the zero has the same offset added.
struct CodeConsts2 {
  uint32_t mask[2], offset[2];
};
__device__ __forceinline__ CodeConsts2 code_consts2() {
  CodeConsts2 c;
  asm volatile("s_mov_b32 %0, %1" : "=s"(c.mask[0]) : "i"(0x000F000Fu));
  asm volatile("s_mov_b32 %0, %1" : "=s"(c.mask[1]) : "i"(0x00F000F0u));
  asm volatile("v_mov_b32 %0, %1" : "=v"(c.offset[0]) : "i"(0x64006400u));
  asm volatile("v_mov_b32 %0, %1" : "=v"(c.offset[1]) : "i"(0x54005400u));
  return c;
}
__device__ __forceinline__ uint32_t pk_add16(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2v, a) + __builtin_bit_cast(half2v, b));
}
__device__ __forceinline__ uint32_t pk_sub16(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2v, a) - __builtin_bit_cast(half2v, b));
}
// pair n of a word minus zeros z0 (1024 + z), z1 (64 + z)
template <int N>
__device__ __forceinline__ uint32_t centred_pair(uint32_t w, uint32_t z0, uint32_t z1,
                                                 const CodeConsts2& cc) {
  return pk_sub16(((N >= 2 ? w >> 8 : w) & cc.mask[N & 1]) | cc.offset[N & 1], N & 1 ? z1 : z0);
}

template <int D, int GS>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(2)))
void k_kv4_attention_wide(Kv4Cache c, Kv4Query a, Partials part) {
  using X = Geo<D, GS>;
  using W = Wide<D, GS>;
  using R = Raw<D, GS>;
  constexpr int NC = W::NC;
  __shared__ __attribute__((aligned(1024))) uint8_t buf0[W::BYTES];
  __shared__ __attribute__((aligned(1024))) uint8_t buf1[W::BYTES];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, q = lane >> 4;
  const Place at = place_of(c, part);
  if (at.tile < 0) return;  // the whole block
  const int b = at.seq, kvh = at.head, split = at.split, tile = at.tile;
  const int group = a.heads / c.kv_heads;
  const int row0 = c.starts[b];
  const int rows = min(min(c.starts[b + 1] - row0, a.max_q), (int)a.n_tokens - row0);
  const int len0 = c.lens[b];
  const int n_cols = rows * group;
  if (tile * W::COLS >= n_cols) return;  // the whole block
  const int P = 1 << c.log2p;
  const int cap = (int)min((int64_t)c.max_blocks << c.log2p, (int64_t)a.max_len);
  const int len = min(len0, cap);
  const int pos0 = len0 - (c.starts[b + 1] - row0);
  const int lo_off = a.window > 0 ? a.window - 1 : 0x3fffffff;

  Column<D, GS> col[NC];
  const int col0 = tile * W::COLS + wave * 16 * NC;
#pragma unroll
  for (int t = 0; t < NC; ++t) {
    const int x = col0 + 16 * t + lr;
    const int i = x / group, h = x - i * group;
    const bool has = x < n_cols;
    const uint16_t* row =
        has ? (const uint16_t*)a.q + (int64_t)(row0 + i) * a.qt + (int64_t)(kvh * group + h) * a.qh
            : nullptr;
    set_query<D, GS>(col[t], read_query<D, GS>(row, q), a.bf16, a.scale);
    col[t].pos = has ? pos0 + i : -1;
  }
  // positions of the block's and of the wave's rows
  const int blk_first = pos0 + tile * W::COLS / group;
  const int blk_last = pos0 + min(tile * W::COLS + W::COLS - 1, n_cols - 1) / group;
  const int first = pos0 + col0 / group;
  const int last = col0 < n_cols ? pos0 + min(col0 + 16 * NC - 1, n_cols - 1) / group : -1;
  int t_lo = max(0, blk_first - lo_off) >> 6, t_hi = max(0, min(len, blk_last + 1) + 63) >> 6;
  {
    const int n = max(0, t_hi - t_lo), s = part.splits;
    const int lo = t_lo + (int)((int64_t)n * split / s), hi = t_lo + (int)((int64_t)n * (split + 1) / s);
    t_lo = lo;
    t_hi = hi;
  }
  const int last_blk = max(0, (len - 1) >> c.log2p);
  const int tt = wave >> 1, sub = wave & 1;  // the wave's decode passes: 32 keys, K result / V piece

  // A lane's keys of a step (K codes, V codes, parameters) and where they lie in a record: key
  // 64 t + x is at (64 t mod P) + (x mod P) of its page.
  const int key_k = 32 * tt + 8 * (lr >> 2) + 4 * sub + (lr & 3), key_v = 32 * tt + 8 * q;
  const int off_k = (key_k & (P - 1)) * (D / 2) + q * (D / 8), off_kz = P * D + 4 * (key_k & (P - 1));
  const int off_v = P * (D / 2) + (key_v & (P - 1)) * (D / 2) + 256 * sub + 16 * lr;
  const int off_vz = P * D + 4 * (P * (X::G + 64 * sub / GS) + (key_v & (P - 1)));
  const int off_p = P * D + 4 * (lane & (P - 1));
  const int32_t* table = c.table + (int64_t)b * c.max_blocks;
  const uint8_t* head_at = c.pages + (int64_t)kvh * c.record;
  const uint32_t page_bytes = (uint32_t)c.kv_heads * (uint32_t)c.record;  // below 2^32
  // their table entries, read one step ahead
  uint32_t page_k, page_v, page_p;
  auto look_up = [&](int t) {
    page_k = table[min((64 * t + key_k) >> c.log2p, last_blk)];
    page_v = table[min((64 * t + key_v) >> c.log2p, last_blk)];
    page_p = table[min((64 * t + lane) >> c.log2p, last_blk)];
  };
  const CodeConsts2 cc = code_consts2();

  // the codes of step t into registers
  auto fetch = [&](R& r, int t) {
    const int base = (64 * t) & (P - 1);
    auto record = [&](uint32_t page, bool& bad) {
      bad = page >= (uint32_t)c.n_pages;
      return head_at + (uint64_t)(bad ? 0u : page) * page_bytes;
    };
    bool bad_k, bad_v, bad_p;
    const uint8_t* rk = record(page_k, bad_k);
    const uint8_t* rv = record(page_v, bad_v);
    const uint8_t* rp = record(page_p, bad_p);
    look_up(t + 1);
    const uint8_t* kp = rk + (off_k + base * (D / 2));
    if constexpr (X::KW == 2) {
      const uint2 w = *(const uint2*)kp;
      r.k[0] = w.x;
      r.k[1] = w.y;
    } else {
      const u32x4 w = *(const u32x4*)kp;
#pragma unroll
      for (int e = 0; e < 4; ++e) r.k[e] = w[e];
    }
    const uint8_t* kz = rk + (off_kz + 4 * base);
#pragma unroll
    for (int g = 0; g < X::G; ++g) r.kz[g] = *(const uint32_t*)(kz + 4 * P * g);
    if (sub < X::H) {
      r.v = *(const u32x4*)(rv + (off_v + base * (D / 2)));
      r.v_there = bad_v ? 0 : len - 64 * t - key_v;
      const uint8_t* vz = rv + (off_vz + 4 * base);
#pragma unroll
      for (int g = 0; g < R::GH; ++g)
#pragma unroll
        for (int i = 0; i < 2; ++i) r.vz[g][i] = *(const u32x4*)(vz + 4 * P * g + 16 * i);
    }
    const uint8_t* pp = rp + (off_p + 4 * base);
#pragma unroll
    for (int k = 0; k < R::PW; ++k) {
      const int pg = wave + kWaves * k;  // side and group
      if (pg < 2 * X::G) r.par[k] = *(const uint32_t*)(pp + 4 * P * pg);
    }
    r.dead = __ballot(bad_p);
  };
  // Keys that do not exist may hold anything.  Their scores are replaced later, whatever they
  // are; their value zeros and steps become zero here.
  auto decode = [&](R& r, int t, uint8_t* buf) -> uint64_t {
    if (r.dead || 64 * t + 64 > len) {
      if (sub < X::H) {
#pragma unroll
        for (int g = 0; g < R::GH; ++g)
#pragma unroll
          for (int e = 0; e < 8; ++e) r.vz[g][e >> 2][e & 3] = e < r.v_there ? r.vz[g][e >> 2][e & 3] : 0u;
      }
      const bool ok = 64 * t + lane < len && !(r.dead >> lane & 1);
#pragma unroll
      for (int k = 0; k < R::PW; ++k) r.par[k] = ok ? r.par[k] : 0u;
    }
    // an infinite step of a key as NaN: its scores could be -infinity, as if it were not there
#pragma unroll
    for (int k = 0; k < R::PW; ++k)
      if (wave + kWaves * k < X::G && (r.par[k] & 0xffffu) == 0x7c00u) r.par[k] |= 0x7e00u;
#pragma unroll
    for (int w = 0; w < X::KW; ++w) {
      const uint32_t par = r.kz[w / X::WPG], zz = __builtin_amdgcn_perm(par, par, 0x03020302u);
      const uint32_t z0 = pk_add16(zz, cc.offset[0]), z1 = pk_add16(zz, cc.offset[1]);
      const u32x4 o = {centred_pair<0>(r.k[w], z0, z1, cc), centred_pair<1>(r.k[w], z0, z1, cc),
                       centred_pair<2>(r.k[w], z0, z1, cc), centred_pair<3>(r.k[w], z0, z1, cc)};
      *(u32x4*)(buf + ((tt * 2 + sub) * X::KW + w) * 1024 + 16 * lane) = o;
    }
    if (sub < X::H) {
      uint32_t z0[R::GH][4], z1[R::GH][4];
#pragma unroll
      for (int g = 0; g < R::GH; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t zz = __builtin_amdgcn_perm(r.vz[g][i >> 1][2 * (i & 1) + 1],
                                                    r.vz[g][i >> 1][2 * (i & 1)], 0x07060302u);
          z0[g][i] = pk_add16(zz, cc.offset[0]);
          z1[g][i] = pk_add16(zz, cc.offset[1]);
        }
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int g = R::GH == 2 ? n >> 1 : 0;
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w = r.v[i];
          o[i] = n == 0   ? centred_pair<0>(w, z0[g][i], z1[g][i], cc)
                 : n == 1 ? centred_pair<1>(w, z0[g][i], z1[g][i], cc)
                 : n == 2 ? centred_pair<2>(w, z0[g][i], z1[g][i], cc)
                          : centred_pair<3>(w, z0[g][i], z1[g][i], cc);
        }
        *(u32x4*)(buf + W::K_BYTES + (tt * X::N + 4 * sub + n) * 1024 + 16 * lane) = o;
      }
    }
#pragma unroll
    for (int k = 0; k < R::PW; ++k) {
      const int pg = wave + kWaves * k;
      if (pg < 2 * X::G) *(uint32_t*)(buf + W::K_BYTES + W::V_BYTES + 256 * pg + 4 * lane) = r.par[k];
    }
    return r.dead;
  };

  uint32_t low = 0;  // the least of the columns' limits
  auto compute = [&](const uint8_t* buf, int t, uint64_t dead) {
    const int key0 = 64 * t;
    if (key0 > last || key0 + 63 < first - lo_off || last < 0) return;  // nothing for this wave
    const bool whole = !dead && key0 + 64 <= len && key0 + 63 <= first && key0 >= last - lo_off;
    const uint8_t* par = buf + W::K_BYTES + W::V_BYTES + 32 * q;
    // scores of all column tiles: an operand read once feeds NC products, and the reads of a
    // result's operands go out before the products of the one before it
    float s[NC][16];
    half8v kk[2][X::KW];
    auto read_k = [&](int hj, half8v (&o)[X::KW]) {
#pragma unroll
      for (int u = 0; u < X::KW; ++u) o[u] = *(const half8v*)(buf + (hj * X::KW + u) * 1024 + 16 * lane);
    };
    read_k(0, kk[0]);
    // products first: one occupies the issue of vector instructions for half of its time, and the
    // other wave of the SIMD fills the rest (prompt 194 -> 188 us)
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int hj = 0; hj < 4; ++hj) {
      const int h = hj >> 1, j = hj & 1;
      if (hj < 3) read_k(hj + 1, kk[(hj + 1) & 1]);
      u32x4 kp[X::G];
#pragma unroll
      for (int g = 0; g < X::G; ++g) kp[g] = *(const u32x4*)(par + 256 * g + 128 * h + 16 * j);
      __builtin_amdgcn_sched_barrier(0);
      f32x4 acc[NC][X::G];
#pragma unroll
      for (int g = 0; g < X::G; ++g)
#pragma unroll
        for (int n = 0; n < NC; ++n) acc[n][g] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < X::WPG; ++u)
#pragma unroll
        for (int g = 0; g < X::G; ++g)
#pragma unroll
          for (int n = 0; n < NC; ++n)
            acc[n][g] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kk[hj & 1][g * X::WPG + u],
                                                               col[n].q[g * X::WPG + u], acc[n][g], 0, 0, 0);
#pragma unroll
      for (int g = 0; g < X::G; ++g)
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int x = 8 * h + 4 * j + e;
            s[n][x] = fmaf(lo16(kp[g][e]), acc[n][g][e], g == 0 ? 0.0f : s[n][x]);
          }
    }
    __builtin_amdgcn_s_setprio(0);
    uint32_t seen[NC];  // bit e: the key of score e exists for the column
#pragma unroll
    for (int n = 0; n < NC; ++n) seen[n] = 0xffff;
    if (!whole) {
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        seen[n] = 0;
        int hi = min(len - 1, col[n].pos) - key0 - 8 * q, lo = col[n].pos - lo_off - key0 - 8 * q;
        asm volatile("" : "+v"(hi), "+v"(lo));  // (keeps the comparisons inside this branch)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int at = e < 8 ? e : e + 24;  // key at + 8 q of the step
          const bool ok = at <= hi && at >= lo && !(dead >> (32 * (e >> 3) + 8 * q) & 1);
          s[n][e] = ok ? s[n][e] : kNegInf;
          seen[n] |= ok ? 1u << e : 0u;
        }
      }
    }
    u32x4 vp[2][X::G][2];
    u16x2 tp = {0, 0};
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int g = 0; g < X::G; ++g)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          vp[h][g][i] = *(const u32x4*)(par + 256 * (X::G + g) + 128 * h + 16 * i);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t w = vp[h][g][i][e];
            tp = __builtin_elementwise_max(tp, __builtin_bit_cast(u16x2, w));
          }
        }
    const uint32_t top = tp[0];
    float mx[NC];
    bool up = top >= low;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      mx[n] = s[n][0];
#pragma unroll
      for (int e = 1; e < 16; ++e) mx[n] = fmaxf(mx[n], s[n][e]);
      mx[n] *= col[n].sigma;
      up |= mx[n] > col[n].m + kSlack;
    }
    if (__any(up)) {
      // the steps that count for each column: finite ones of keys that it sees.  Read from LDS once more,
      // so that the loop over all tiles keeps its registers (prompt of 4096 tokens: 194 us from vp, 187 so)
      uint32_t most[NC];
#pragma unroll
      for (int n = 0; n < NC; ++n) most[n] = top;
      if (!whole) {
        u16x2 t[NC];
#pragma unroll
        for (int n = 0; n < NC; ++n) t[n] = u16x2{0, 0};
#pragma unroll 1
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 8; e += 2)
#pragma unroll
            for (int g = 0; g < X::G; ++g) {
              const uint2 v = *(const uint2*)(par + 256 * (X::G + g) + 128 * h + 4 * e);
#pragma unroll
              for (int n = 0; n < NC; ++n)
                t[n] = __builtin_elementwise_max(
                    t[n], __builtin_bit_cast(u16x2, step_pair(v.x, v.y) & seen_halves(seen[n] >> (8 * h), e)));
            }
#pragma unroll
        for (int n = 0; n < NC; ++n) most[n] = max(t[n][0], t[n][1]);
      }
      low = 0xffffu;
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        Column<D, GS>& cl = col[n];
        uint32_t all = most[n];
        if (__any(all >= 0x7c00u)) {  // NaN or infinite: the largest of the others
          all = 0;
#pragma unroll 1
          for (int x = 0; x < 16 * X::G; ++x) {
            const uint32_t v = *(const uint32_t*)(par + 256 * (X::G + (x >> 4)) + 128 * (x >> 3 & 1) + 4 * (x & 7));
            all = max(all, counted_step(v, seen[n] >> (x & 15) & 1));
          }
        }
        all = max(all, (uint32_t)__shfl_xor((int)all, 16));
        all = max(all, (uint32_t)__shfl_xor((int)all, 32));
        cl.limit = limit_above(all, cl.limit);
        low = min(low, cl.limit);
        const float m = fmaxf(cl.m, max_q(mx[n]));
        const float nM = m == kNegInf ? 0.0f : weight_exponent(cl.limit) - m;
        const float x = cl.m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(nM - cl.nM);
        cl.m = m;
        cl.nM = nM;
        cl.l *= x;
#pragma unroll
        for (int i = 0; i < X::N; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) cl.o[i][e] *= x;
      }
    }
    u32x4 w[NC][2][X::G];
#pragma unroll
    for (int n = 0; n < NC; ++n) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        s[n][e] = __builtin_amdgcn_exp2f(fmaf(s[n][e], col[n].sigma, col[n].nM));
        col[n].l += s[n][e];
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int g = 0; g < X::G; ++g)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t pa = vp[h][g][i >> 1][2 * (i & 1)], pb = vp[h][g][i >> 1][2 * (i & 1) + 1];
            w[n][h][g][i] = pair16(fmaf(s[n][8 * h + 2 * i], lo16(pa), 0.0f),
                                   fmaf(s[n][8 * h + 2 * i + 1], lo16(pb), 0.0f));
          }
    }
    if (!whole) {  // a masked key's step may be NaN
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t bits = (seen[n] >> (8 * h + 2 * i) & 1 ? 0xffffu : 0u) |
                                  (seen[n] >> (8 * h + 2 * i + 1) & 1 ? 0xffff0000u : 0u);
#pragma unroll
            for (int g = 0; g < X::G; ++g) w[n][h][g][i] &= bits;
          }
    }
    constexpr int PV = 2 * X::N / 4;  // groups of four value operands, each read a group ahead
    half8v vv[2][4];
    auto read_v = [&](int g, half8v (&o)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = *(const half8v*)(buf + W::K_BYTES + (4 * g + i) * 1024 + 16 * lane);
    };
    read_v(0, vv[0]);
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int g = 0; g < PV; ++g) {
      if (g + 1 < PV) read_v(g + 1, vv[(g + 1) & 1]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int h = (4 * g + i) / X::N, o = (4 * g + i) % X::N;
#pragma unroll
        for (int n = 0; n < NC; ++n)
          col[n].o[o] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
              vv[g & 1][i], __builtin_bit_cast(half8v, w[n][h][o / (GS / 16)]), col[n].o[o], 0, 0, 0);
      }
    }
    __builtin_amdgcn_s_setprio(0);
  };

  if (t_lo < t_hi) {
    R r;
    look_up(t_lo);
    fetch(r, t_lo);
    uint64_t dead = decode(r, t_lo, buf0);
    __syncthreads();
    for (int t = t_lo; t < t_hi; t += 2) {
      if (t + 1 < t_hi) fetch(r, t + 1);
      compute(buf0, t, dead);
      if (t + 1 >= t_hi) break;
      dead = decode(r, t + 1, buf1);
      __syncthreads();
      if (t + 2 < t_hi) fetch(r, t + 2);
      compute(buf1, t + 1, dead);
      if (t + 2 >= t_hi) break;
      dead = decode(r, t + 2, buf0);
      __syncthreads();
    }
  }

#pragma unroll
  for (int t = 0; t < NC; ++t) {
    const int x = col0 + 16 * t + lr;
    Column<D, GS>& cl = col[t];
    cl.l = sum_q(cl.l);
    if (x < n_cols) {
      const int i = x / group, h = x - i * group;
      const int64_t r = (int64_t)(row0 + i) * a.heads + kvh * group + h;
      const bool join = part.splits > 1;
      const float inv = join ? 1.0f : cl.l == 0.0f ? 0.0f : 1.0f / cl.l;
#pragma unroll
      for (int n = 0; n < X::N; ++n) {
        const int ch = 16 * n + 4 * q;
        if (join) {
          *(f32x4*)(part.o + (r * part.splits + split) * D + ch) = cl.o[n];
        } else {
          const float v[4] = {cl.o[n][0] * inv, cl.o[n][1] * inv, cl.o[n][2] * inv, cl.o[n][3] * inv};
          store4(a.out, r * D + ch, a.bf16, v);
        }
      }
      if (q == 0) {
        if (join) {
          part.ml[(r * part.splits + split) * 2] = cl.M();
          part.ml[(r * part.splits + split) * 2 + 1] = cl.l;
        } else if (a.lse) {
          a.lse[r] = lse_of(cl.M(), cl.l);
        }
      }
    }
  }
}

// Joins the splits of a (token, head): D / 4 threads a row and part, part w adds splits w,
// w + PARTS, ... in order, then the parts are added in order.
template <int D, int PARTS, bool DIVIDED>
__global__ __launch_bounds__(256) void k_kv4_join(Kv4Cache c, Kv4Query a, Partials part,
                                                  int64_t n_rows) {
  constexpr int T = D / 4, ROWS = 256 / (T * PARTS);
  __shared__ f32x4 so[PARTS > 1 ? PARTS : 1][T];
  __shared__ float sm[PARTS], sl[PARTS];
  const int x = threadIdx.x % T, w = threadIdx.x / T % PARTS;
  const int64_t r = (int64_t)block_number() * ROWS + threadIdx.x / (T * PARTS);
  if (r >= n_rows) return;  // (one row a block, or no barrier)
  const int64_t t = r / a.heads;
  int64_t first = r * part.splits, step = 1;  // slots
  int S = part.splits;
  if constexpr (DIVIDED) {
    const int b = kv4_sequence(c, t);
    if (b < 0 || t - c.starts[b] >= a.max_q) return;  // (one row a block, or no barrier)
    const int group = a.heads / c.kv_heads, h = (int)(r - t * a.heads), kvh = h / group;
    const int2 p = *(const int2*)(part.parts + 2 * ((int64_t)b * c.kv_heads + kvh));
    if (p.y == 1) return;
    S = p.y;
    step = 16;
    first = ((int64_t)kvh * (part.splits + c.n_seqs) + p.x) * 16 + (t - c.starts[b]) * group + h - kvh * group;
  }
  // wide: read before it is known whether the row has partials (what is read is workspace either way)
  const float2* ml = (const float2*)part.ml + first;
  const float* po = part.o + first * D + 4 * x;
  float M = kNegInf, l = 0.0f;
#pragma unroll 4
  for (int s = w; s < S; s += PARTS) M = fmaxf(M, ml[s * step].x);
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = w; s < S; s += PARTS) {
    const float2 y = ml[s * step];
    const f32x4 v = *(const f32x4*)(po + s * step * D);
    const float k = y.x == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(y.x - M);
    l = fmaf(y.y, k, l);
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = fmaf(v[e], k, o[e]);
  }
  if constexpr (PARTS > 1) {
    so[w][x] = o;
    if (x == 0) {
      sm[w] = M;
      sl[w] = l;
    }
    __syncthreads();
    if (w > 0) return;
    float all = M;
#pragma unroll
    for (int i = 1; i < PARTS; ++i) all = fmaxf(all, sm[i]);
    l = 0.0f;
    o = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
      const float k = sm[i] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(sm[i] - all);
      l = fmaf(sl[i], k, l);
      const f32x4 v = so[i][x];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = fmaf(v[e], k, o[e]);
    }
    M = all;
  }
  if constexpr (!DIVIDED) {  // a row past a sequence's bound has no partials
    const int b = kv4_sequence(c, t);
    if (b < 0 || t - c.starts[b] >= a.max_q) return;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const float v[4] = {o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv};
  store4(a.out, r * D + 4 * x, a.bf16, v);
  if (x == 0 && a.lse) a.lse[r] = lse_of(M, l);
}

template <int D, bool DIVIDED>
hipError_t launch_join(const Kv4Cache& c, const Kv4Query& q, const Partials& part, int64_t rows,
                       hipStream_t stream) {
  constexpr int kParts = 1024 / D, kRows = 1024 / D;
  // many parts a row
  if (part.splits / (DIVIDED ? c.n_seqs : 1) >= 16)
    hipLaunchKernelGGL((k_kv4_join<D, kParts, DIVIDED>), grid_of(rows), dim3(256), 0, stream, c, q,
                       part, rows);
  else
    hipLaunchKernelGGL((k_kv4_join<D, 1, DIVIDED>), grid_of((rows + kRows - 1) / kRows), dim3(256), 0,
                       stream, c, q, part, rows);
  return hipGetLastError();
}

template <int D, int GS>
hipError_t launch_dg(const Kv4Cache& c, const Kv4Query& q, const Kv4Plan& p, const Partials& part,
                     int64_t rows, hipStream_t stream) {
  const int64_t blocks = kv4_blocks(p, c.n_seqs, c.kv_heads);
  if (blocks > kMaxBlocks) return hipErrorInvalidValue;
  const dim3 grid = grid_of(blocks);
  if (p.wide)
    hipLaunchKernelGGL((k_kv4_attention_wide<D, GS>), grid, dim3(64 * kWaves), 0, stream, c, q, part);
  else if (p.splits > 1)
    hipLaunchKernelGGL((k_kv4_attention<D, GS, kWaves, true>), grid, dim3(64 * kWaves), 0, stream, c, q, part);
  else if (p.waves == 8)
    hipLaunchKernelGGL((k_kv4_attention<D, GS, 8, false>), grid, dim3(512), 0, stream, c, q, part);
  else
    hipLaunchKernelGGL((k_kv4_attention<D, GS, kWaves, false>), grid, dim3(64 * kWaves), 0, stream, c, q, part);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits <= 1) return e;
  return p.wide ? launch_join<D, false>(c, q, part, rows, stream) : launch_join<D, true>(c, q, part, rows, stream);
}

}  // namespace

// Keys beyond which few columns are divided whatever the number of sequences.
constexpr int64_t kUndivided = 5120;

Kv4Plan kv4_plan(int64_t n_seqs, int heads, int kv_heads, int dim, int group, int64_t max_q,
                 int64_t max_len, int64_t window) {
  Kv4Plan p;
  const int64_t cols = max_q * (heads / kv_heads);
  const int64_t keys = window > 0 && window < max_len ? std::min(max_len, window + max_q) : max_len;
  p.wide = cols > 16;
  p.waves = kWaves;
  if (p.wide) {
    const int64_t per = 16 * wide_tiles(dim, group) * kWaves;
    p.tiles = (int)((cols + per - 1) / per);
    const int64_t blocks = n_seqs * kv_heads * p.tiles;
    // Keys split up to two blocks a compute unit, at least 256 keys a split (512 tokens after 7680
    // others, 32 heads on 8: 232 us unsplit, 98 so; 64 after 1984: 75 and 25; three chunks over a
    // window, 480 blocks: 96 and 94, with twice as many splits 100).
    const int64_t s = std::min((512 + blocks - 1) / blocks, (keys + 255) / 256);
    p.splits = (int)std::max<int64_t>(s, 1);
    return p;
  }
  p.tiles = 1;
  p.splits = 1;
  const int64_t blocks = n_seqs * kv_heads;
  // Dividing the keys over two blocks a compute unit (one sequence of 131072 tokens: 39 us with 512
  // blocks, 42 with 1024, 65 with 4096) costs a second launch and a start for each part of a
  // sequence; it pays once sequences are long for their number.  8 key heads of 128, lengths from
  // a quarter of the largest to the largest, undivided and divided: one sequence of 1024 tokens
  // 11.9 and 11.7 us, of 4096 27.2 and 12.5; 8 sequences up to 2048 16.9 and 19.0, up to 3072
  // 22.0 and 19.9; 32 up to 4096 31.2 and 33.1, up to 6144 40.7 and 40.0; 64 up to 4096 46.4 and
  // 46.9, up to 8192 87.8 and 84.7; 256 up to 8192 291 and 288.
  if (keys > std::min(1024 + 20 * blocks, kUndivided) && blocks <= 2048 &&
      n_seqs * (keys / 32 + 2) < ((int64_t)1 << 30))
    p.splits = std::max(512 / kv_heads, 1);
  // Undivided: eight waves a block where the blocks are no more than the compute units (32
  // sequences up to 2048 tokens: 22.1 us with four, 20.2 with eight), else four (64: 28.7 and 34.5).
  else if (blocks <= 256)
    p.waves = 8;
  return p;
}

namespace {

// slots of partial sums
int64_t kv4_slots(const Kv4Plan& p, int64_t n_tokens, int64_t n_seqs, int heads, int kv_heads) {
  return p.wide ? n_tokens * heads * p.splits : (int64_t)kv_heads * (p.splits + n_seqs) * 16;
}

}  // namespace

size_t kv4_workspace(const Kv4Plan& p, int64_t n_tokens, int64_t n_seqs, int heads, int kv_heads, int dim) {
  if (p.splits <= 1) return 0;
  return (size_t)kv4_slots(p, n_tokens, n_seqs, heads, kv_heads) * (dim + 2) * sizeof(float) +
         (p.wide ? 0 : (size_t)n_seqs * kv_heads * 2 * sizeof(int32_t));
}

size_t kv4_workspace_any_window(int64_t n_tokens, int64_t n_seqs, int heads, int kv_heads, int dim,
                                int group, int64_t max_q, int64_t max_len) {
  auto of = [&](int64_t keys) {
    return kv4_workspace(kv4_plan(n_seqs, heads, kv_heads, dim, group, max_q, keys, 0), n_tokens, n_seqs,
                         heads, kv_heads, dim);
  };
  // A window is a smaller bound on the keys.  The parts of the wide form grow with that bound.  Few
  // columns have one number of parts or none, and none also where the tiles are too many to count, so
  // that a window may divide what the whole length does not: the fewest keys that are divided in any
  // case (or all) decide that.
  return std::max(of(max_len), of(std::min(max_len, kUndivided + 1)));
}

hipError_t launch_kv4_attention(const Kv4Cache& c, const Kv4Query& q, const Kv4Plan& p,
                                void* workspace, hipStream_t stream) {
  const int64_t rows = q.n_tokens * q.heads;
  if (rows <= 0 || c.n_seqs <= 0) return hipSuccess;
  const int64_t slots = kv4_slots(p, q.n_tokens, c.n_seqs, q.heads, c.kv_heads);
  Partials part;
  part.splits = p.splits;
  part.tiles = p.tiles;
  part.o = (float*)workspace;
  part.ml = part.o + slots * c.dim;
  part.parts = (int32_t*)(part.ml + slots * 2);
  switch (c.dim * 1000 + c.group) {
    case 64032: return launch_dg<64, 32>(c, q, p, part, rows, stream);
    case 64064: return launch_dg<64, 64>(c, q, p, part, rows, stream);
    case 128032: return launch_dg<128, 32>(c, q, p, part, rows, stream);
    case 128064: return launch_dg<128, 64>(c, q, p, part, rows, stream);
    case 128128: return launch_dg<128, 128>(c, q, p, part, rows, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace awq
