// Write and read-back of the 4-bit key/value cache.
//
// Pages: "AWQ" scholia-log notes §2.3, §3.2 (the group quantiser); kwkr.cn §1.2, §2.1 (codes
// with an fp16 step a group).
//
// A row (token, head) is D / 8 lanes of 8 consecutive channels, for keys and values alike; a
// group's range is reduced across its g / 8 lanes.  Bound by reading the fp16 rows from HBM
// (4 bytes in for 1 byte of codes out).
#include <hip/hip_runtime.h>

#include "int8_quant.h"
#include "kv4_cache.h"

namespace awq {

namespace {

// Codes (nibble e = channel e) and the parameter pair of the lane's group.
template <int LANES>
__device__ __forceinline__ uint32_t quantise_group(const float (&v)[8], bool zp, uint32_t& par) {
  float code[8], step, zero;
  quantize8<LANES>(v, 4, zp, code, step, zero);
  float odd = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) odd = fabsf(v[i]) < __builtin_inff() ? odd : 1.0f;
  odd = group_max<LANES>(odd);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) w |= (uint32_t)(int)code[i] << (4 * i);
  par = (uint32_t)f2h(step) | ((uint32_t)f2h(zero) << 16);
  if (odd != 0.0f) {
    w = 0;
    par = 0x7e00u;  // step NaN, zero 0
  }
  return w;
}

template <bool BF16, int D, int GS>
__global__ __launch_bounds__(256) void k_kv4_append(Kv4Cache c, const uint16_t* __restrict__ k,
                                                    int64_t kt, int64_t kh,
                                                    const uint16_t* __restrict__ v, int64_t vt,
                                                    int64_t vh, int64_t n_rows) {
  constexpr int LPR = D / 8, G = D / GS;
  const int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LPR;
  const int l = threadIdx.x % LPR;
  if (row >= n_rows) return;  // whole rows: the lanes of a group leave together
  const int64_t t = row / c.kv_heads;
  const int head = (int)(row - t * c.kv_heads);
  float x[2][8];
  load_row8<BF16, true>(k + t * kt + head * kh, nullptr, kFoldNone, 8 * l, D, x[0]);
  load_row8<BF16, true>(v + t * vt + head * vh, nullptr, kFoldNone, 8 * l, D, x[1]);
  const int b = kv4_sequence(c, t);
  if (b < 0) return;
  const int pos = c.lens[b] - (c.starts[b + 1] - (int)t);
  const int64_t at = kv4_record_at(c, b, pos, head);
  if (at < 0) return;
  uint8_t* rec = c.pages + at;
  const int P = 1 << c.log2p, p = pos & (P - 1);
  uint32_t kp, vp;
  const uint32_t kw = quantise_group<GS / 8>(x[0], c.zero_point, kp);
  const uint32_t vw = quantise_group<GS / 8>(x[1], c.zero_point, vp);
  // K: the lane's 8 channels are one word
  const int j = 8 * l / GS, ing = 8 * l % GS;
  const int q = ing / (GS / 4), u = ing % (GS / 4) / 8;
  *(uint32_t*)(rec + p * (D / 2) + q * (D / 8) + j * (GS / 8) + u * 4) = kw;
  // V: channel 16 n + r of a token is nibble n mod 4 of its half-word (n / 4, r).  The lane
  // holds n = l / 2 for the 8 r of its parity; with the words of the other three n of the same
  // n / 4 (lanes 2, 4 and 6 away) it assembles two of those 8 halves.
  uint32_t w4[4];
  const int c4 = (l >> 1) & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) w4[i] = (uint32_t)__shfl_xor((int)vw, 2 * (i ^ c4));
  uint8_t* vb = rec + P * (D / 2) + (p >> 3) * (D * 4) + (l >> 3) * 256 + ((p & 7) >> 1) * 4 + (p & 1) * 2;
#pragma unroll
  for (int e = 2 * c4; e < 2 * c4 + 2; ++e) {
    uint32_t h = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) h |= ((w4[i] >> (4 * e)) & 15u) << (4 * i);
    *(uint16_t*)(vb + (8 * (l & 1) + e) * 16) = (uint16_t)h;
  }
  if (ing == 0) {
    uint32_t* par = (uint32_t*)(rec + P * D);
    par[j * P + p] = kp;
    par[(G + j) * P + p] = vp;
  }
}

template <bool BF16, int D, int GS>
__global__ __launch_bounds__(256) void k_kv4_read(Kv4Cache c, uint16_t* __restrict__ k,
                                                  uint16_t* __restrict__ v, int64_t n_rows) {
  constexpr int LPR = D / 8, G = D / GS;
  const int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LPR;
  const int l = threadIdx.x % LPR;
  if (row >= n_rows) return;
  const int64_t t = row / c.kv_heads;
  const int head = (int)(row - t * c.kv_heads);
  uint4 ko = {0u, 0u, 0u, 0u}, vo = {0u, 0u, 0u, 0u};
  const int b = kv4_sequence(c, t);
  const int pos = b < 0 ? -1 : c.lens[b] - (c.starts[b + 1] - (int)t);
  const int64_t at = b < 0 ? -1 : kv4_record_at(c, b, pos, head);
  if (at >= 0) {
    const uint8_t* rec = c.pages + at;
    const int P = 1 << c.log2p, p = pos & (P - 1);
    const int j = 8 * l / GS, ing = 8 * l % GS;
    const int q = ing / (GS / 4), u = ing % (GS / 4) / 8;
    const uint32_t kw = *(const uint32_t*)(rec + p * (D / 2) + q * (D / 8) + j * (GS / 8) + u * 4);
    const uint8_t* vb =
        rec + P * (D / 2) + (p >> 3) * (D * 4) + (l >> 3) * 256 + ((p & 7) >> 1) * 4 + (p & 1) * 2;
    const uint32_t* par = (const uint32_t*)(rec + P * D);
    const uint32_t kp = par[j * P + p], vp = par[(G + j) * P + p];
    const float ks = h2f((uint16_t)kp), kz = h2f((uint16_t)(kp >> 16));
    const float vs = h2f((uint16_t)vp), vz = h2f((uint16_t)(vp >> 16));
    uint16_t kr[8], vr[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t h = *(const uint16_t*)(vb + (8 * (l & 1) + e) * 16);
      const int kc = (kw >> (4 * e)) & 15, vc = (h >> (4 * ((l >> 1) & 3))) & 15;
      kr[e] = to16<BF16>(((float)kc - kz) * ks);
      vr[e] = to16<BF16>(((float)vc - vz) * vs);
    }
    __builtin_memcpy(&ko, kr, 16);
    __builtin_memcpy(&vo, vr, 16);
  }
  *(uint4*)(k + row * D + 8 * l) = ko;
  *(uint4*)(v + row * D + 8 * l) = vo;
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
  const int64_t rows = n_tokens * c.kv_heads, blocks = (rows * (c.dim / 8) + 255) / 256;
  if (rows <= 0) return hipSuccess;
  if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
#define AWQ_APPEND(B, D, GS)                                                                   \
  hipLaunchKernelGGL((k_kv4_append<B, D, GS>), dim3((unsigned)blocks), dim3(256), 0, stream, c, \
                     (const uint16_t*)k, kt, kh, (const uint16_t*)v, vt, vh, rows)
  if (bf16) { AWQ_KV4_DG(AWQ_APPEND, true) } else { AWQ_KV4_DG(AWQ_APPEND, false) }
#undef AWQ_APPEND
  return hipGetLastError();
}

hipError_t launch_kv4_read(const Kv4Cache& c, int64_t n_tokens, bool bf16, void* k, void* v,
                           hipStream_t stream) {
  const int64_t rows = n_tokens * c.kv_heads, blocks = (rows * (c.dim / 8) + 255) / 256;
  if (rows <= 0) return hipSuccess;
  if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
#define AWQ_READ(B, D, GS)                                                                    \
  hipLaunchKernelGGL((k_kv4_read<B, D, GS>), dim3((unsigned)blocks), dim3(256), 0, stream, c, \
                     (uint16_t*)k, (uint16_t*)v, rows)
  if (bf16) { AWQ_KV4_DG(AWQ_READ, true) } else { AWQ_KV4_DG(AWQ_READ, false) }
#undef AWQ_READ
  return hipGetLastError();
}

}  // namespace awq
