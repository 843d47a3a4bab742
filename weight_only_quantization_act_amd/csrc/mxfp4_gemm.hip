// Product in MXFP4: y[t][m] = sum_i x[t][i] w[m][i] + bias[m], both operands blocks of 32 4-bit
// floating-point elements with a power of two each.
//
// Pages: "AWQ" scholia-log notes §1.1 (the layer's product); "AWQ量化技术解析" (kwkr.cn) §4.2
// (dequantisation fused into the product): here the matrix cores take the codes and the scales as
// they are.  An instruction adds 64 or 128 products of 4-bit elements (exact, multiples of 1/4 times a
// power of two) and the running fp32 sum with one rounding.
//
// Tiles (many tokens): as for 8-bit integers, a block computes BT tokens x BM outputs from stages of 128 bytes of
// K (256 columns) that move global -> LDS by DMA into a ring of NS (rows of 128 bytes, the 16-byte
// chunk index XOR-swizzled with the row).  v_mfma_scale_f32_32x32x64_f8f6f4 takes, in lane l, one block of row l
// mod 32 of both operands and its scale byte.  Which columns an instruction multiplies is free as
// long as both operands agree: step k of a stage takes block 4 (l div 32) + k, so that a lane's
// four scales of a stage are one 32-bit word of the scales' layout, byte k of it chosen by the
// instruction.  The words of a tile's rows are contiguous ([column word][row]) and come
// by DMA as well.  Element e of the result is row 8 (e div 4) + 4 (l div 32) + e mod 4 of the first operand
// (token), column l mod 32 of the second (output).  Rows past the matrices and chunks past K arrive as
// zeros, or as scales of rows that are dropped.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "grid.h"
#include "int8_quant.h"
#include "mfma_dma.h"
#include "mx_format.h"
#include "mx_internal.h"
#include "mxfp4_plan.h"
#include "serve_internal.h"

namespace awq {

namespace {

typedef int int32x8 __attribute__((ext_vector_type(8)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr int kFp4 = 4;  // the instruction's code for the format e2m1

__device__ __forceinline__ int32x8 operand(const int32x4& a) {  // 32 elements; the rest is not read
  return int32x8{a[0], a[1], a[2], a[3], 0, 0, 0, 0};
}

template <int BT_, int BM_, int WT_, int WM_, int NS_>
struct MxTile {
  static constexpr int BT = BT_, BM = BM_, WT = WT_, WM = WM_, NS = NS_;
  static constexpr int BK = 128;  // bytes of K a stage
  static constexpr int WAVES = WT * WM, THREADS = 64 * WAVES;
  static constexpr int TI = BT / WT / 32, MI = BM / WM / 32;
  static constexpr int X_BYTES = BT * BK, CODES = (BT + BM) * BK;
  static constexpr int XS_BYTES = 2 * 4 * BT, BYTES = CODES + 2 * 4 * (BT + BM);
  static constexpr int DMA_X = X_BYTES / 1024 / WAVES, DMA_W = BM * BK / 1024 / WAVES;
  // scales: DMAs of 64 words; where they do not divide evenly a wave repeats another's
  static constexpr int S_X = 2 * BT / 64, S_ALL = 2 * (BT + BM) / 64;
  static constexpr int DMA_S = (S_ALL + WAVES - 1) / WAVES;
  static constexpr int PER = DMA_X + DMA_W + DMA_S;
  static_assert(DMA_X >= 1 && DMA_W >= 1 && S_X >= 1, "each wave loads a part of both operands");
  static_assert(TI >= 1 && MI >= 1, "each wave has a 32 x 32 tile at least");
  __device__ static int swz(int row) { return (row & 7) ^ ((row >> 3) & 1); }
};

// splits > 1: block z sums its share of K and stores the fp32 tile to part [splits][T][M].
template <class S, bool BF16>
__global__ __launch_bounds__(S::THREADS) void k_mxfp4_tiles(MxArgs a, int tiles_t, int tiles_m,
                                                            int splits, float* __restrict__ part) {
  constexpr int NS = S::NS;
  __shared__ __attribute__((aligned(1024))) uint8_t sm[NS * S::BYTES];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63;
  const int wt = wave / S::WM, wm = wave % S::WM;

  // Blocks go to the 8 XCDs in turn; renumbered so that each XCD walks a contiguous range of
  // tiles in bands of 8 token tiles, whose panels its compute units share in that XCD's L2.
  constexpr int kBand = 8;
  const int total = tiles_t * tiles_m;
  const int b = (int)block_number(), xcd = b & 7, local = b >> 3;
  if (b >= total) return;  // the whole block
  const int q8 = total >> 3, r8 = total & 7;
  const int logical = xcd < r8 ? xcd * (q8 + 1) + local : r8 * (q8 + 1) + (xcd - r8) * q8 + local;
  const int band = logical / (kBand * tiles_m);
  const int band_rows = min(kBand, tiles_t - band * kBand);
  const int in_band = logical - band * kBand * tiles_m;
  const int tt = band * kBand + in_band % band_rows, tm = in_band / band_rows;
  const int t0 = tt * S::BT, m0 = tm * S::BM;

  const int rows_x = min(S::BT, a.T - t0), rows_w = min(S::BM, a.M - m0);
  const int ldx = (int)a.ldx, ldw = (int)a.ldw;  // a panel of rows spans less than 2^31 bytes
  // the last row ends at byte KB (its allocation may end there)
  const int32x4 rx = buffer_rsrc(a.x + (int64_t)t0 * a.ldx, (unsigned)(rows_x - 1) * ldx + a.KB);
  const int32x4 rw = buffer_rsrc(a.w + (int64_t)m0 * a.ldw, (unsigned)(rows_w - 1) * ldw + a.KB);

  // A wave-DMA fills 8 rows of 128 bytes: lane l its row l / 8, physical chunk l % 8, which
  // holds logical chunk (l % 8) ^ swz(row).  swz depends on row mod 16, so on the parity of
  // the 8-row block as well as on the lane.
  constexpr unsigned kOut = 0x80000000u;
  const int dr = lane >> 3;
  const int ce = (lane & 7) ^ S::swz(dr), co = (lane & 7) ^ S::swz(dr + 8);
  const unsigned row_x = wave * S::DMA_X * 8 + dr, row_w = wave * S::DMA_W * 8 + dr;
  const unsigned ldsb = lds_address(sm);
  // 128-byte steps of this split: kt0 .. kt1 - 1, walked in whole turns of the ring
  const int steps = (a.KB + S::BK - 1) / S::BK, z = blockIdx.z;
  const int kt0 = (int)((int64_t)steps * z / splits);
  const int n_steps = (int)((int64_t)steps * (z + 1) / splits) - kt0;
  const int nk = (n_steps + NS - 1) / NS * NS;
  const int words = (a.KB + 63) >> 6;  // scale words a row

  auto dma = [&](int st, int kt) {
    const int k0 = (kt0 + kt) * S::BK;
    const bool in = kt < n_steps;
    const bool oke = in && k0 + ce * 16 < a.KB, oko = in && k0 + co * 16 < a.KB;
#pragma unroll
    for (int j = 0; j < S::DMA_X; ++j) {
      const bool odd = (wave * S::DMA_X + j) & 1;
      const unsigned r = row_x + 8 * j;
      const unsigned v = (odd ? oko : oke) && r < (unsigned)rows_x
                             ? r * ldx + (odd ? co : ce) * 16 : kOut;
      lds_dma16(rx, ldsb + st * S::BYTES + (wave * S::DMA_X + j) * 1024u, v, k0);
    }
#pragma unroll
    for (int j = 0; j < S::DMA_W; ++j) {
      const bool odd = (wave * S::DMA_W + j) & 1;
      const unsigned r = row_w + 8 * j;
      const unsigned v = (odd ? oko : oke) && r < (unsigned)rows_w
                             ? r * ldw + (odd ? co : ce) * 16 : kOut;
      lds_dma16(rw, ldsb + st * S::BYTES + S::X_BYTES + (wave * S::DMA_W + j) * 1024u, v, k0);
    }
    // scale words 2 kt and 2 kt + 1 of the tile's rows: [2][BT], then [2][BM]
    const int q0 = 2 * (kt0 + kt);
    const int nq = in ? min(2, words - q0) : 0;
#pragma unroll
    for (int j = 0; j < S::DMA_S; ++j) {
      const int d = (wave * S::DMA_S + j) % S::S_ALL;
      const bool is_x = d < S::S_X;
      const int64_t ld = is_x ? a.ldxs : a.ldws;
      const uint32_t* base = (is_x ? a.xs + t0 : a.ws + m0) + (nq > 0 ? (int64_t)q0 * ld : 0);
      const int rows = is_x ? rows_x : rows_w;
      const int32x4 rs = buffer_rsrc(base, nq > 0 ? ((unsigned)(nq - 1) * (unsigned)ld + rows) * 4u : 0u);
      const int i = (is_x ? d : d - S::S_X) * 64 + lane, n = is_x ? S::BT : S::BM;
      const int q = i / n, r = i % n;
      const unsigned v = q < nq && r < rows ? ((unsigned)q * (unsigned)ld + r) * 4u : kOut;
      lds_dma4(rs, ldsb + st * S::BYTES + S::CODES + d * 256u, v);
    }
  };

  const int fr = lane & 31, fh = lane >> 5, fs = S::swz(fr);
  const int x_off = (wt * S::TI * 32 + fr) * S::BK;
  const int w_off = S::X_BYTES + (wm * S::MI * 32 + fr) * S::BK;
  const int xs_off = S::CODES + (fh * S::BT + wt * S::TI * 32 + fr) * 4;
  const int ws_off = S::CODES + S::XS_BYTES + (fh * S::BM + wm * S::MI * 32 + fr) * 4;
  struct Frag {
    int32x4 x[S::TI], w[S::MI];
  };
  struct Scales {
    int x[S::TI], w[S::MI];
  };
  auto load = [&](const uint8_t* base, int ks, Frag& f) {
    const int chunk = ((4 * fh + ks) ^ fs) * 16;
#pragma unroll
    for (int i = 0; i < S::TI; ++i) f.x[i] = *(const int32x4*)(base + x_off + i * 32 * S::BK + chunk);
#pragma unroll
    for (int i = 0; i < S::MI; ++i) f.w[i] = *(const int32x4*)(base + w_off + i * 32 * S::BK + chunk);
  };
  auto load_scales = [&](const uint8_t* base, Scales& s) {
#pragma unroll
    for (int i = 0; i < S::TI; ++i) s.x[i] = *(const int*)(base + xs_off + i * 128);
#pragma unroll
    for (int i = 0; i < S::MI; ++i) s.w[i] = *(const int*)(base + ws_off + i * 128);
  };
  floatx16 acc[S::TI][S::MI];
#pragma unroll
  for (int i = 0; i < S::TI; ++i)
#pragma unroll
    for (int j = 0; j < S::MI; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  auto mma = [&](auto ks, const Frag& f, const Scales& s) {
    constexpr int B = decltype(ks)::value;
#pragma unroll
    for (int i = 0; i < S::TI; ++i)
#pragma unroll
      for (int j = 0; j < S::MI; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            operand(f.x[i]), operand(f.w[j]), acc[i][j], kFp4, kFp4, B, s.x[i], B, s.w[j]);
  };
  using std::integral_constant;

  // NS stages in flight; a stage is refilled after the barrier that follows its last fragment
  // read, and the DMAs past the end of K read zeros into a slot nobody uses, so the number in
  // flight, hence the vmcnt to wait for, is constant.
  Frag f0, f1;
  Scales sc, sn;
  auto step = [&](int st, int kt) {
    const uint8_t* cur = sm + st * S::BYTES;
    const uint8_t* next = sm + (st + 1) % NS * S::BYTES;
    load(cur, 1, f1);
    mma(integral_constant<int, 0>{}, f0, sc);
    load(cur, 2, f0);
    mma(integral_constant<int, 1>{}, f1, sc);
    load(cur, 3, f1);
    mma(integral_constant<int, 2>{}, f0, sc);
    __builtin_amdgcn_s_waitcnt(WaitVmLgkm0<(NS - 2) * S::PER>::value);  // stage kt + 1 has landed
    __builtin_amdgcn_s_barrier();
    dma(st, kt + NS);
    load_scales(next, sn);
    load(next, 0, f0);
    mma(integral_constant<int, 3>{}, f1, sc);
    sc = sn;
  };
  if (nk > 0) {
#pragma unroll
    for (int st = 0; st < NS; ++st) dma(st, st);
    __builtin_amdgcn_s_waitcnt(WaitVmLgkm0<(NS - 1) * S::PER>::value);
    __builtin_amdgcn_s_barrier();
    load_scales(sm, sc);
    load(sm, 0, f0);
    for (int kt = 0; kt < nk; kt += NS) {
#pragma unroll
      for (int st = 0; st < NS; ++st) step(st, kt + st);
    }
    __builtin_amdgcn_s_waitcnt(WaitVmLgkm0<0>::value);  // no LDS write may outlive the block
  }

  if (splits > 1) {
    float* dst = part + (int64_t)z * a.T * a.M;
#pragma unroll
    for (int j = 0; j < S::MI; ++j)
#pragma unroll
      for (int i = 0; i < S::TI; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int m = m0 + (wm * S::MI + j) * 32 + (lane & 31);
          const int t = t0 + (wt * S::TI + i) * 32 + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
          if (t < a.T && m < a.M) dst[(int64_t)t * a.M + m] = acc[i][j][e];
        }
    return;
  }
  const uint16_t* bias = (const uint16_t*)a.bias;
  uint16_t* y = (uint16_t*)a.y;
#pragma unroll
  for (int j = 0; j < S::MI; ++j) {
    const int m = m0 + (wm * S::MI + j) * 32 + (lane & 31);
    const bool mok = m < a.M;
    const float bs = mok && bias ? from16<BF16>(bias[m]) : 0.0f;
#pragma unroll
    for (int i = 0; i < S::TI; ++i) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int t = t0 + (wt * S::TI + i) * 32 + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
        if (t < a.T && mok) {
          float v = acc[i][j][e];
          if (bias) v = v + bs;
          y[(int64_t)t * a.ldy + m] = to16<BF16>(v);
        }
      }
    }
  }
}

// The sum of the splits' tiles in their order.  Four outputs a thread where M allows it.
template <bool BF16, int V>
__global__ __launch_bounds__(256) void k_mxfp4_finish(MxArgs a, int splits,
                                                      const float* __restrict__ part) {
  typedef float fvec __attribute__((ext_vector_type(V)));
  const int64_t n = (int64_t)a.T * a.M;
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V;
  if (i >= n) return;
  const int t = (int)(i / a.M), m = (int)(i - (int64_t)t * a.M);
  fvec s = *(const fvec*)(part + i);
  for (int z = 1; z < splits; ++z) s += *(const fvec*)(part + z * n + i);
  const uint16_t* bias = (const uint16_t*)a.bias;
  uint16_t* y = (uint16_t*)a.y + (int64_t)t * a.ldy + m;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    float v = s[e];
    if (bias) v = v + from16<BF16>(bias[m + e]);
    y[e] = to16<BF16>(v);
  }
}

// ---- few tokens --------------------------------------------------------------------------
//
// Up to 16 tokens the product is bound by reading the weights once.  A block takes 16 RT outputs
// and all tokens; its eight waves take 256-byte pieces of K (512 columns) in turn.  The weights go
// from memory to the operand registers of v_mfma_scale_f32_16x16x128_f8f6f4 directly: lane l has
// row l mod 16 and the 64 bytes from 64 (l div 16) of a piece, whose four blocks' scales are one word;
// instruction u takes block u of each lane.  The next piece's loads are ahead of the products of
// this one; the tokens' operands come from L2.  The waves' fp32 sums are added through LDS in their
// order.  Result element e of lane l is output 4 (l div 16) + e, token l mod 16.
//
// FUSED: the block first quantises the tokens into LDS, with the first weights already on their way;
// every block repeats that (a few thousand values from L2) in place of a launch before this one.
constexpr int kFewWaves = 8;

struct MxFewArgs {
  MxArgs g;
  const uint16_t* x16;  // FUSED: the tokens, their scales, columns and row stride
  const float* s;
  int64_t ldx16;
  int cols;
  bool vec;
};

template <int RT, bool FUSED, bool BF16>
__global__ __launch_bounds__(64 * kFewWaves) void k_mxfp4_few(MxFewArgs f) {
  const MxArgs& a = f.g;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];  // FUSED: codes [T][pieces 256], words [T][4 pieces]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, q = lane >> 4;
  const unsigned first = block_number() * 16u * RT;  // below 2^32 past M, too
  if (first >= (unsigned)a.M) return;                // the whole block
  const int m0 = (int)first;
  const int nch = (a.KB + 255) >> 8;
  const int words = (a.KB + 63) >> 6;

  // rows past the last repeat it and are dropped; blocks past K read the row's start and count 0
  struct Piece {
    int32x4 w[RT][4];
    int s[RT];
  };
  const uint8_t* wrow[RT];
  const uint32_t* srow[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int row = min(m0 + 16 * r + lr, a.M - 1);
    wrow[r] = a.w + (int64_t)row * a.ldw;
    srow[r] = a.ws + row;
  }
  auto load_w = [&](Piece& o, int ch) {
    const int k = ch * 256 + 64 * q;
    const int word = 4 * ch + q;
#pragma unroll
    for (int r = 0; r < RT; ++r) o.s[r] = (int)srow[r][(int64_t)(word < words ? word : 0) * a.ldws];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool in = k + 16 * u < a.KB;
#pragma unroll
      for (int r = 0; r < RT; ++r) o.w[r][u] = *(const int32x4*)(wrow[r] + (in ? k + 16 * u : 0));
    }
  };
  Piece p0, p1;
  if (wave < nch) load_w(p0, wave);

  uint32_t* lwords = (uint32_t*)(lds + (size_t)a.T * nch * 256);
  if constexpr (FUSED) {
    const int n8 = nch * 64;  // 8-column chunks of whole pieces
    for (int i = tid; i < a.T * n8; i += 64 * kFewWaves) {
      const int t = i / n8, ch = i - t * n8;  // sixteen lanes have one token and one word
      float v[8];
      const uint16_t* row = f.x16 + t * f.ldx16;
      const int fold = f.s ? kFoldDivide : kFoldNone;
      if (f.vec) load_row8<BF16, true>(row, f.s, fold, 8 * ch, f.cols, v);
      else load_row8<BF16, false>(row, f.s, fold, 8 * ch, f.cols, v);
      uint32_t byte;
      const uint32_t c = mx_codes8(v, byte);
      *(uint32_t*)(lds + (size_t)t * nch * 256 + 4 * ch) = c;
      const uint32_t w = mx_scale_word(byte);
      if ((ch & 15) == 0) lwords[t * nch * 4 + (ch >> 4)] = w;
    }
    __syncthreads();
  }

  // columns past the last token repeat it and are dropped
  const int tok = min(lr, a.T - 1);
  floatx4 acc[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) acc[r] = floatx4{0.f, 0.f, 0.f, 0.f};
  struct XPiece {
    int32x4 x[4];
    int s;
  };
  auto load_x = [&](XPiece& o, int ch) {
    const int k = ch * 256 + 64 * q;
    const int word = 4 * ch + q;
    if constexpr (FUSED) {
      o.s = (int)lwords[tok * nch * 4 + word];
#pragma unroll
      for (int u = 0; u < 4; ++u) o.x[u] = *(const int32x4*)(lds + (size_t)tok * nch * 256 + k + 16 * u);
    } else {
      o.s = (int)a.xs[(int64_t)(word < words ? word : 0) * a.ldxs + tok];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        o.x[u] = *(const int32x4*)(a.x + (int64_t)tok * a.ldx + (k + 16 * u < a.KB ? k + 16 * u : 0));
    }
  };
  auto piece = [&](Piece& w, XPiece& x, int ch) {
    if (ch == nch - 1) {  // blocks past K count nothing (their scales may be any row's)
      const int k = ch * 256 + 64 * q;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (k + 16 * u >= a.KB) {
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            w.w[r][u] = int32x4{0, 0, 0, 0};
            w.s[r] = w.s[r] & ~(255 << (8 * u));
          }
          x.s = x.s & ~(255 << (8 * u));
        }
    }
    auto step = [&](auto uu) {
      constexpr int u = decltype(uu)::value;
#pragma unroll
      for (int r = 0; r < RT; ++r)
        acc[r] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            operand(w.w[r][u]), operand(x.x[u]), acc[r], kFp4, kFp4, u, w.s[r], u, x.s);
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
  };
  // a piece's tokens are asked for before the next piece's weights: loads return in order, so
  // waiting for the tokens does not wait for those weights
  for (int ch = wave; ch < nch; ch += 2 * kFewWaves) {
    XPiece x;
    load_x(x, ch);
    if (ch + kFewWaves < nch) load_w(p1, ch + kFewWaves);
    __builtin_amdgcn_sched_barrier(0);
    piece(p0, x, ch);
    if (ch + kFewWaves >= nch) break;
    load_x(x, ch + kFewWaves);
    if (ch + 2 * kFewWaves < nch) load_w(p0, ch + 2 * kFewWaves);
    __builtin_amdgcn_sched_barrier(0);
    piece(p1, x, ch + kFewWaves);
  }

  // the waves' sums, then one (tile, lane) a thread
  __shared__ floatx4 sum[kFewWaves][RT][64];
#pragma unroll
  for (int r = 0; r < RT; ++r) sum[wave][r][lane] = acc[r];
  __syncthreads();
  const uint16_t* bias = (const uint16_t*)a.bias;
  for (int i = tid; i < RT * 64; i += 64 * kFewWaves) {
    const int tile = i >> 6, l = i & 63;
    floatx4 v = sum[0][tile][l];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) {
      const floatx4 o = sum[w][tile][l];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += o[e];
    }
    const int t = l & 15, m = m0 + 16 * tile + 4 * (l >> 4);
    if (t >= a.T) continue;
    uint16_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (m + e < a.M) {
        float y = v[e];
        if (bias) y = y + from16<BF16>(bias[m + e]);
        o[e] = to16<BF16>(y);
      }
    }
    uint16_t* y = (uint16_t*)a.y + (int64_t)t * a.ldy + m;
    if (m + 4 <= a.M && a.ldy % 4 == 0 && ((uintptr_t)a.y & 7) == 0) {
      uint2 p;
      p.x = o[0] | ((uint32_t)o[1] << 16);
      p.y = o[2] | ((uint32_t)o[3] << 16);
      *(uint2*)y = p;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (m + e < a.M) y[e] = o[e];
    }
  }
}

template <class S, bool BF16>
hipError_t launch_tiles(const MxArgs& a, int splits, float* part, hipStream_t stream) {
  const int tt = (a.T + S::BT - 1) / S::BT, tm = (a.M + S::BM - 1) / S::BM;
  const int64_t tiles = (int64_t)tt * tm;
  if (tiles > kMaxBlocks) return hipErrorInvalidValue;
  dim3 grid = grid_of(tiles);
  grid.z = (unsigned)splits;
  hipLaunchKernelGGL((k_mxfp4_tiles<S, BF16>), grid, dim3(S::THREADS), 0, stream, a, tt, tm, splits,
                     part);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits <= 1) return e;
  const int64_t n = (int64_t)a.T * a.M;
  if (a.M % 4 == 0)
    hipLaunchKernelGGL((k_mxfp4_finish<BF16, 4>), dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0,
                       stream, a, splits, part);
  else
    hipLaunchKernelGGL((k_mxfp4_finish<BF16, 1>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0,
                       stream, a, splits, part);
  return hipGetLastError();
}

template <int RT, bool FUSED>
hipError_t launch_few(const MxFewArgs& f, hipStream_t stream) {
  const dim3 grid = grid_of((f.g.M + 16 * RT - 1) / (16 * RT)), block(64 * kFewWaves);
  const size_t lds = FUSED ? (size_t)f.g.T * ((f.g.KB + 255) / 256) * (256 + 16) : 0;
  if (f.g.bf16)
    hipLaunchKernelGGL((k_mxfp4_few<RT, FUSED, true>), grid, block, lds, stream, f);
  else
    hipLaunchKernelGGL((k_mxfp4_few<RT, FUSED, false>), grid, block, lds, stream, f);
  return hipGetLastError();
}

template <bool BF16>
hipError_t launch_plan(const MxArgs& a, const MxPlan& p, float* part, hipStream_t stream) {
  switch (p.form) {
    case kMxTile32: return launch_tiles<MxTile<32, 128, 1, 4, 3>, BF16>(a, p.splits, part, stream);
    case kMxTile64: return launch_tiles<MxTile<64, 128, 2, 2, 3>, BF16>(a, p.splits, part, stream);
    case kMxTile128: return launch_tiles<MxTile<128, 128, 2, 2, 2>, BF16>(a, p.splits, part, stream);
    default: return launch_tiles<MxTile<256, 256, 2, 4, 2>, BF16>(a, 1, nullptr, stream);
  }
}

}  // namespace

size_t mxfp4_matmul_workspace(int64_t T, int64_t M, int64_t KB) {
  const MxPlan p = mxfp4_plan(T, M, KB);
  return p.splits > 1 ? (size_t)p.splits * T * M * sizeof(float) : 0;
}

hipError_t launch_mxfp4_matmul(const MxArgs& a, void* workspace, hipStream_t stream) {
  if (a.T <= 0 || a.M <= 0) return hipSuccess;
  const MxPlan p = mxfp4_plan(a.T, a.M, a.KB);
  if (p.form == kMxFew) {
    const MxFewArgs f{a, nullptr, nullptr, 0, 0, false};
    return mxfp4_few_rows(a.M) == 2 ? launch_few<2, false>(f, stream) : launch_few<1, false>(f, stream);
  }
  return a.bf16 ? launch_plan<true>(a, p, (float*)workspace, stream)
                : launch_plan<false>(a, p, (float*)workspace, stream);
}

bool mxfp4_linear_fused(int64_t T, int64_t M, int64_t cols) { return T == 1 && cols <= 65536; }

hipError_t launch_mxfp4_linear_fused(const MxArgs& a, const void* x, int64_t ldx, const float* s,
                                     int cols, hipStream_t stream) {
  if (a.T <= 0 || a.M <= 0) return hipSuccess;
  const MxFewArgs f{a, (const uint16_t*)x, s, ldx, cols, row_vector_loads(x, a.T > 1 ? ldx : 0, s)};
  return mxfp4_few_rows(a.M) == 2 ? launch_few<2, true>(f, stream) : launch_few<1, true>(f, stream);
}

}  // namespace awq
