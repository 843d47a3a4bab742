// Write and read-back of the 4-bit key/value cache.
//
// Pages: "AWQ" scholia-log notes §2.3, §3.2 (the group quantiser); kwkr.cn §1.2, §2.1 (codes
// with an fp16 step a group).
//
// A row (token, head) is D / 8 lanes of 8 consecutive channels, for keys and values alike; a
// group's range is reduced across its g / 8 lanes.  Value codes change their order through LDS
// (a word of the record holds four channels, 16 apart, of two tokens): written one by one they
// would be quarter words scattered over the record (prompts of up to 8191 tokens, 8 heads of 128:
// 94 us for write and read-back so, 58 us through LDS).  Bound by the 16-bit rows on the HBM side
// (4 bytes for 1 byte of codes) and, in the write, by the quantiser's vector instructions: 27000
// tokens of 8 heads are written in 35 us (4.1 TB/s) and read back in 23 us (6.1 TB/s).
// Four heads a block in place of one, to share the search for a block's rows, measured the same.
#include <hip/hip_runtime.h>

#include "grid.h"
#include "int8_quant.h"
#include "kv4_cache.h"

namespace awq {

namespace {

// a / b from y = RN(1 / b), while nothing underflows: the residual a - b q of the product q = a y is
// exact in one fused multiply-add (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990), so that the last one rounds a / b to within 2^-23 of an ulp.  That
// is RN(a / b) unless a / b lies that near the middle of two floats.  For b = 15 or 7 none does
// (1 / 30 of an ulp at least).  Of the other quotients only rint is used, so only those near
// k + 1/2, k < 16, count: for a 16-bit a they come that near the middle beside k + 1/2 only with a =
// S (k + 1/2), S of few bits, and b one ulp beside S, and then only for b of all mantissa bits.
__device__ __forceinline__ float quotient(float a, float b, float y) {
  const float q = a * y;
  return fmaf(fmaf(-q, b, a), y, q);
}

// Codes (nibble e = channel e) and the parameter pair of the lane's group, from eight 16-bit
// values: the quantiser of quantizer.h (4 bits, no channel scales) with the same results.  Values
// of 16 bits tie often (a wave of them nearly always somewhere), so the quotients are all
// corrected, without its test for half-integers and division behind a branch (write of 27000
// tokens, 8 heads: 39 us with the test, 35 without and with ZP a template argument).
template <bool BF16, int LANES, bool ZP>
__device__ __forceinline__ uint32_t quantise_group(const uint4 raw, uint32_t& par) {
  const uint32_t r[4] = {raw.x, raw.y, raw.z, raw.w};
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = from16<BF16>(r[i] & 0xffffu);
    v[2 * i + 1] = BF16 ? __builtin_bit_cast(float, r[i] & 0xffff0000u) : from16<BF16>(r[i] >> 16);
  }
  // NaN or infinity in the lane: the largest pattern without the sign
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  u16x2 big = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    big = __builtin_elementwise_max(big, __builtin_bit_cast(u16x2, r[i] & 0x7fff7fffu));
  const bool odd = max(big[0], big[1]) >= (BF16 ? 0x7f80 : 0x7c00);
  float hi = 0.0f, lo = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    hi = fmaxf(hi, ZP ? v[i] : fabsf(v[i]));
    lo = fminf(lo, v[i]);
  }
  hi = group_max<LANES>(odd ? __builtin_inff() : hi);
  lo = ZP ? group_min<LANES>(lo) : 0.0f;
  const float range = hi - lo, top = ZP ? 15.0f : 7.0f;
  float st = quotient(range, top, ZP ? 1.0f / 15.0f : 1.0f / 7.0f);
  // what the corrected quotients do not cover: steps whose residuals may underflow, and those of
  // all mantissa bits (whose reciprocal one step of Newton's need not round correctly either)
  const uint32_t bits = __builtin_bit_cast(uint32_t, st);
  const bool rare = st < 0x1p-90f || (bits & 0x7fffffu) == 0x7fffffu;
  float q[8], z;
  if (rare) {
    st = range / top;
    if (st == 0.0f) st = 1.0f;
    z = rintf(-lo / st);
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = rintf(v[i] / st);
  } else {
    const float y0 = __builtin_amdgcn_rcpf(st);
    const float y = fmaf(fmaf(-st, y0, 1.0f), y0, y0);
    z = rintf(quotient(-lo, st, y));
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = rintf(quotient(v[i], st, y));
  }
  z = ZP ? fminf(fmaxf(z, 0.0f), 15.0f) : 8.0f;
  float code[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    code[i] = ZP ? fminf(fmaxf(q[i] + z, 0.0f), 15.0f) : fminf(fmaxf(q[i], -7.0f), 7.0f) + 8.0f;
  // four codes at a time as one exact number below 2^16
  uint32_t half[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    half[h] = (uint32_t)fmaf(fmaf(fmaf(code[4 * h + 3], 16.0f, code[4 * h + 2]), 16.0f, code[4 * h + 1]), 16.0f,
                             code[4 * h]);
  par = (uint32_t)f2h(st) | ((uint32_t)f2h(z) << 16);
  if (!(range < __builtin_inff())) {
    par = 0x7e00u;  // step NaN, zero 0
    return 0;
  }
  return half[0] | (half[1] << 16);
}

// Which rows a block works on: R = 2048 / D consecutive positions of one sequence, the first a
// multiple of R, so that a block's value codes are whole 8-token blocks of the record.
// Sequence s owns the R-row groups from starts[s] / R + 2 s on: that leaves it enough of them
// wherever its first position lies, without a sum over the sequences before it.  The groups
// after the last sequence's hold the rows that belong to none.
template <int D>
struct Rows {
  static constexpr int R = 2048 / D;
  int seq, pos0, t0;  // sequence (-1: none), position and row index of the block's first row
  int first, end;     // rows of the sequence: first <= t < end
};
template <int D>
__device__ __forceinline__ Rows<D> rows_of(const Kv4Cache& c, int blk, int n_tokens) {
  constexpr int R = Rows<D>::R;
  const auto* starts = (const __attribute__((address_space(4))) int32_t*)(uintptr_t)c.starts;
  Rows<D> r;
  const int n = c.n_seqs;
  auto own = [&](int s) { return starts[s] / R + 2 * s; };
  if (blk >= own(n)) {
    r.seq = -1;
    r.pos0 = 0;
    r.t0 = starts[n] + (blk - own(n)) * R;
    r.first = starts[n];
    r.end = n_tokens;
    return r;
  }
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (own(mid) <= blk) lo = mid; else hi = mid - 1;
  }
  r.seq = lo;
  r.first = starts[lo];
  r.end = min(starts[lo + 1], n_tokens);
  const int p = c.lens[lo] - (starts[lo + 1] - r.first);  // position of the first row
  r.pos0 = (p & ~(R - 1)) + (blk - own(lo)) * R;
  r.t0 = r.first + (r.pos0 - p);
  return r;
}

// Where the 32-bit word of value codes w of a block's R positions lies in the record (the block
// is whole 8-token blocks: words in the record's order), and its two tokens' rows.
template <int D>
__device__ __forceinline__ int value_word_row(int w) { return (w / D) * 8 + 2 * (w & 3); }

template <bool BF16, int D, int GS, bool ZP>
__global__ __launch_bounds__(256) void k_kv4_append(Kv4Cache c, const uint16_t* __restrict__ k,
                                                    int64_t kt, int64_t kh,
                                                    const uint16_t* __restrict__ v, int64_t vt,
                                                    int64_t vh, int n_tokens) {
  constexpr int LPR = D / 8, G = D / GS, R = Rows<D>::R;
  __shared__ uint32_t vwords[R][LPR + 1];
  __shared__ int64_t page_at[R];  // each row's record, or -1
  const int number = (int)block_number();
  const int group = number / c.kv_heads, head = number - group * c.kv_heads;
  if (group > n_tokens / Rows<D>::R + 2 * c.n_seqs) return;  // the whole block
  const Rows<D> rows = rows_of<D>(c, group, n_tokens);
  if (rows.seq < 0 || rows.t0 >= rows.end || rows.t0 + R <= rows.first) return;  // the whole block
  const int row = threadIdx.x / LPR, l = threadIdx.x % LPR;
  const int P = 1 << c.log2p;
  {
    const int t = rows.t0 + row, pos = rows.pos0 + row;
    const bool in = t >= rows.first && t < rows.end;
    uint4 xk = {0u, 0u, 0u, 0u}, xv = xk;
    if (in) {  // asked for before the table's answer is waited for
      xk = *(const uint4*)(k + t * kt + head * kh + 8 * l);
      xv = *(const uint4*)(v + t * vt + head * vh + 8 * l);
    }
    const int64_t at = in ? kv4_record_at(c, rows.seq, pos, head) : -1;
    if (l == 0) page_at[row] = at;
    if (at >= 0) {  // the lanes of a row alike
      const int p = pos & (P - 1);
      const int j = 8 * l / GS, ing = 8 * l % GS;
      const int q = ing / (GS / 4), u = ing % (GS / 4) / 8;
      uint8_t* rec = c.pages + at;
      uint32_t kp, vp;
      const uint32_t kw = quantise_group<BF16, GS / 8, ZP>(xk, kp);
      vwords[row][l] = quantise_group<BF16, GS / 8, ZP>(xv, vp);
      // keys: the lane's 8 channels are one word
      *(uint32_t*)(rec + p * (D / 2) + q * (D / 8) + j * (GS / 8) + u * 4) = kw;
      if (ing == 0) {
        uint32_t* par = (uint32_t*)(rec + P * D);
        par[j * P + p] = kp;
        par[(G + j) * P + p] = vp;
      }
    }
  }
  __syncthreads();
  // values: a thread assembles words of the record, two tokens of four channels 16 apart each
  // (the two lie in one page)
#pragma unroll
  for (int w = threadIdx.x; w < R * D / 8; w += 256) {
    const int r0 = value_word_row<D>(w), h = w % D / 64, r = w % 64 / 4;
    const int64_t at0 = page_at[r0], at1 = page_at[r0 + 1];
    if (at0 < 0 && at1 < 0) continue;
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int n = 0; n < 4; ++n)
        word |= ((vwords[r0 + e][2 * (4 * h + n) + (r >> 3)] >> (4 * (r & 7))) & 15u) << (16 * e + 4 * n);
    uint8_t* dst = c.pages + (at0 < 0 ? at1 : at0) + P * (D / 2) +
                   (((rows.pos0 + r0) & (P - 1)) >> 3) * (D * 4) + (w % D) * 4;
    if (at0 >= 0 && at1 >= 0) *(uint32_t*)dst = word;
    else if (at0 >= 0) *(uint16_t*)dst = (uint16_t)word;
    else *(uint16_t*)(dst + 2) = (uint16_t)(word >> 16);
  }
}

template <bool BF16, int D, int GS>
__global__ __launch_bounds__(256) void k_kv4_read(Kv4Cache c, uint16_t* __restrict__ k,
                                                  uint16_t* __restrict__ v, int n_tokens) {
  constexpr int LPR = D / 8, G = D / GS, R = Rows<D>::R;
  __shared__ uint32_t words[R * D / 8];
  const int number = (int)block_number();
  const int group = number / c.kv_heads, head = number - group * c.kv_heads;
  if (group > n_tokens / Rows<D>::R + 2 * c.n_seqs) return;  // the whole block
  const Rows<D> rows = rows_of<D>(c, group, n_tokens);
  if (rows.t0 >= rows.end || rows.t0 + R <= rows.first) return;  // the whole block
  const int P = 1 << c.log2p;
  if (rows.seq >= 0) {
    // the value codes of the block's positions, coalesced (those of other tokens unused)
#pragma unroll
    for (int w = threadIdx.x; w < R * D / 8; w += 256) {
      const int pos = rows.pos0 + value_word_row<D>(w);
      const int64_t at = kv4_record_at(c, rows.seq, pos, head);
      words[w] = at < 0 ? 0u
                        : *(const uint32_t*)(c.pages + at + P * (D / 2) +
                                             ((pos & (P - 1)) >> 3) * (D * 4) + (w % D) * 4);
    }
  }
  __syncthreads();
  const int row = threadIdx.x / LPR, l = threadIdx.x % LPR;
  const int t = rows.t0 + row, pos = rows.pos0 + row;
  if (t < rows.first || t >= rows.end) return;
  uint4 ko = {0u, 0u, 0u, 0u}, vo = {0u, 0u, 0u, 0u};
  const int64_t at = rows.seq < 0 ? -1 : kv4_record_at(c, rows.seq, pos, head);
  if (at >= 0) {
    const uint8_t* rec = c.pages + at;
    const int p = pos & (P - 1);
    const int j = 8 * l / GS, ing = 8 * l % GS;
    const int q = ing / (GS / 4), u = ing % (GS / 4) / 8;
    const uint32_t kw = *(const uint32_t*)(rec + p * (D / 2) + q * (D / 8) + j * (GS / 8) + u * 4);
    const uint32_t* par = (const uint32_t*)(rec + P * D);
    const uint32_t kp = par[j * P + p], vp = par[(G + j) * P + p];
    const float ks = h2f((uint16_t)kp), kz = h2f((uint16_t)(kp >> 16));
    const float vs = h2f((uint16_t)vp), vz = h2f((uint16_t)(vp >> 16));
    uint16_t kr[8], vr[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t word = words[(row >> 3) * D + (l >> 3) * 64 + (8 * (l & 1) + e) * 4 + ((row & 7) >> 1)];
      const int kc = (kw >> (4 * e)) & 15, vc = (word >> (16 * (row & 1) + 4 * ((l >> 1) & 3))) & 15;
      kr[e] = to16<BF16>(((float)kc - kz) * ks);
      vr[e] = to16<BF16>(((float)vc - vz) * vs);
    }
    __builtin_memcpy(&ko, kr, 16);
    __builtin_memcpy(&vo, vr, 16);
  }
  const int64_t o = ((int64_t)t * c.kv_heads + head) * D + 8 * l;
  *(uint4*)(k + o) = ko;
  *(uint4*)(v + o) = vo;
}

}  // namespace

#define AWQ_KV4_DG(F, BF)                                        \
  switch (c.dim * 1000 + c.group) {                              \
    case 64032: F(BF, 64, 32); break;                            \
    case 64064: F(BF, 64, 64); break;                            \
    case 128032: F(BF, 128, 32); break;                          \
    case 128064: F(BF, 128, 64); break;                          \
    case 128128: F(BF, 128, 128); break;                         \
    default: return hipErrorInvalidValue;                        \
  }

hipError_t launch_kv4_append(const Kv4Cache& c, const void* k, int64_t kt, int64_t kh,
                             const void* v, int64_t vt, int64_t vh, int64_t n_tokens, bool bf16,
                             hipStream_t stream) {
  if (n_tokens <= 0) return hipSuccess;
  const int64_t blocks = kv4_store_blocks(n_tokens, c.dim, c.n_seqs, c.kv_heads);
  if (blocks > kMaxBlocks) return hipErrorInvalidValue;
#define AWQ_APPEND_Z(B, D, GS, Z)                                                              \
  hipLaunchKernelGGL((k_kv4_append<B, D, GS, Z>), grid_of(blocks), dim3(256), 0, stream, c, \
                     (const uint16_t*)k, kt, kh, (const uint16_t*)v, vt, vh, (int)n_tokens)
#define AWQ_APPEND(B, D, GS)                              \
  if (c.zero_point) { AWQ_APPEND_Z(B, D, GS, true); }     \
  else { AWQ_APPEND_Z(B, D, GS, false); }
  if (bf16) { AWQ_KV4_DG(AWQ_APPEND, true) } else { AWQ_KV4_DG(AWQ_APPEND, false) }
#undef AWQ_APPEND
#undef AWQ_APPEND_Z
  return hipGetLastError();
}

hipError_t launch_kv4_read(const Kv4Cache& c, int64_t n_tokens, bool bf16, void* k, void* v,
                           hipStream_t stream) {
  if (n_tokens <= 0) return hipSuccess;
  const int64_t blocks = kv4_store_blocks(n_tokens, c.dim, c.n_seqs, c.kv_heads);
  if (blocks > kMaxBlocks) return hipErrorInvalidValue;
  const dim3 grid = grid_of(blocks);
#define AWQ_READ(B, D, GS)                                                     \
  hipLaunchKernelGGL((k_kv4_read<B, D, GS>), grid, dim3(256), 0, stream, c, (uint16_t*)k, \
                     (uint16_t*)v, (int)n_tokens)
  if (bf16) { AWQ_KV4_DG(AWQ_READ, true) } else { AWQ_KV4_DG(AWQ_READ, false) }
#undef AWQ_READ
  return hipGetLastError();
}

}  // namespace awq
