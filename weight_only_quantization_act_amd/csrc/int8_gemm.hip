// Product in 8-bit integers: y[t][m] = float(sum_i x[t][i] w[m][i]) xstep[t] wstep[m] + bias[m].
//
// Pages: "AWQ" scholia-log notes §2.3 (symmetric integer quantiser); the product is exact in
// int32, so neither the order of the sum nor a split of it changes a result.
//
// Tiles (many tokens): both operands are K-contiguous bytes.  A block computes BT tokens x BM
// outputs from tiles of 128 bytes of K, which move global -> LDS by DMA into a ring of NS
// stages (rows of 128 bytes, the 16-byte chunk index XOR-swizzled with the row, so that the
// fragment reads of 32 rows are free of bank conflicts), and feeds
// v_mfma_i32_32x32x32_i8: lane l supplies 16 bytes of row l mod 32 at chunk 2 k + l div 32 for
// both operands; element e of the result is row 8 (e div 4) + 4 (l div 32) + e mod 4 of the
// first operand (token), column l mod 32 of the second (output).  Rows past the matrices and
// chunks past K lie outside the buffer resources or take an out-of-range offset and arrive as
// zeros.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "grid.h"
#include "int8_plan.h"
#include "int8_quant.h"
#include "mfma_dma.h"
#include "serve_internal.h"

namespace awq {

namespace {

// y = (float(acc) xstep) wstep + bias, each operation rounded once in fp32, then to 16 bits.
__device__ __forceinline__ float scaled(int acc, float xs, float ws) {
  return (float)acc * xs * ws;
}

template <int BT_, int BM_, int WT_, int WM_, int NS_>
struct Tile {
  static constexpr int BT = BT_, BM = BM_, WT = WT_, WM = WM_, NS = NS_;
  static constexpr int BK = 128;  // bytes of K a stage
  static constexpr int WAVES = WT * WM, THREADS = 64 * WAVES;
  static constexpr int TI = BT / WT / 32, MI = BM / WM / 32;
  static constexpr int X_BYTES = BT * BK, BYTES = (BT + BM) * BK;
  static constexpr int DMA_X = X_BYTES / 1024 / WAVES, DMA_W = BM * BK / 1024 / WAVES;
  static constexpr int KSTEPS = BK / 32;
  static_assert(DMA_X >= 1 && DMA_W >= 1, "each wave loads a part of both operands");
  static_assert(TI >= 1 && MI >= 1, "each wave has a 32 x 32 tile at least");
  __device__ static int swz(int row) { return (row & 7) ^ ((row >> 3) & 1); }
};

// Bound by the matrix cores: 256 x 256 tiles on sixteen waves of 128 x 32, one block a compute
// unit, do 8192 tokens through 28672 x 8192 in 1.70 ms, 2.27 Pop/s (128 x 128 tiles, two blocks a
// compute unit, 2.19 ms).  Small tiles keep more blocks for fewer tokens (int8_plan.h).
//
// splits > 1: block z sums its share of K and stores the int32 tile to part [splits][T][M].
template <class S, bool BF16>
__global__ __launch_bounds__(S::THREADS) void k_int8_tiles(Int8Args a, int tiles_t, int tiles_m,
                                                           int splits, int* __restrict__ part) {
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
  // the last row ends at column K (its allocation may end there)
  const int32x4 rx = buffer_rsrc(a.x + (int64_t)t0 * a.ldx, (unsigned)(rows_x - 1) * ldx + a.K);
  const int32x4 rw = buffer_rsrc(a.w + (int64_t)m0 * a.ldw, (unsigned)(rows_w - 1) * ldw + a.K);

  // A wave-DMA fills 8 rows of 128 bytes: lane l its row l / 8, physical chunk l % 8, which
  // holds logical chunk (l % 8) ^ swz(row).  swz depends on row mod 16, so on the parity of
  // the 8-row block as well as on the lane.
  constexpr unsigned kOut = 0x80000000u;
  const int dr = lane >> 3;
  const int ce = (lane & 7) ^ S::swz(dr), co = (lane & 7) ^ S::swz(dr + 8);
  const unsigned row_x = wave * S::DMA_X * 8 + dr, row_w = wave * S::DMA_W * 8 + dr;
  const unsigned ldsb = lds_address(sm);
  // 128-byte steps of this split: kt0 .. kt1 - 1, walked in whole turns of the ring
  const int steps = (a.K + S::BK - 1) / S::BK, z = blockIdx.z;
  const int kt0 = (int)((int64_t)steps * z / splits);
  const int n_steps = (int)((int64_t)steps * (z + 1) / splits) - kt0;
  const int nk = (n_steps + NS - 1) / NS * NS;

  auto dma = [&](int st, int kt) {
    const int k0 = (kt0 + kt) * S::BK;
    const bool in = kt < n_steps;
    const bool oke = in && k0 + ce * 16 < a.K, oko = in && k0 + co * 16 < a.K;
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
  };

  const int fr = lane & 31, fh = lane >> 5, fs = S::swz(fr);
  const int x_off = (wt * S::TI * 32 + fr) * S::BK;
  const int w_off = S::X_BYTES + (wm * S::MI * 32 + fr) * S::BK;
  struct Frag {
    int32x4 x[S::TI], w[S::MI];
  };
  auto load = [&](const uint8_t* base, int ks, Frag& f) {
    const int chunk = ((2 * ks + fh) ^ fs) * 16;
#pragma unroll
    for (int i = 0; i < S::TI; ++i) f.x[i] = *(const int32x4*)(base + x_off + i * 32 * S::BK + chunk);
#pragma unroll
    for (int i = 0; i < S::MI; ++i) f.w[i] = *(const int32x4*)(base + w_off + i * 32 * S::BK + chunk);
  };
  int32x16 acc[S::TI][S::MI];
#pragma unroll
  for (int i = 0; i < S::TI; ++i)
#pragma unroll
    for (int j = 0; j < S::MI; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;
  auto mma = [&](const Frag& f) {
#pragma unroll
    for (int i = 0; i < S::TI; ++i)
#pragma unroll
      for (int j = 0; j < S::MI; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.x[i], f.w[j], acc[i][j], 0, 0, 0);
  };

  // NS stages in flight; a stage is refilled after the barrier that follows its last fragment
  // read, and the DMAs past the end of K read zeros into a slot nobody uses, so the number in
  // flight, hence the vmcnt to wait for, is constant.
  constexpr int PER = S::DMA_X + S::DMA_W;
  Frag f0, f1;
  auto step = [&](int st, int kt) {
    const uint8_t* cur = sm + st * S::BYTES;
    const uint8_t* next = sm + (st + 1) % NS * S::BYTES;
#pragma unroll
    for (int ks = 0; ks + 2 < S::KSTEPS; ks += 2) {
      load(cur, ks + 1, f1);
      mma(f0);
      load(cur, ks + 2, f0);
      mma(f1);
    }
    load(cur, S::KSTEPS - 1, f1);
    mma(f0);
    __builtin_amdgcn_s_waitcnt(WaitVmLgkm0<(NS - 2) * PER>::value);  // stage kt + 1 has landed
    __builtin_amdgcn_s_barrier();
    dma(st, kt + NS);
    load(next, 0, f0);
    mma(f1);
  };
  if (nk > 0) {
#pragma unroll
    for (int st = 0; st < NS; ++st) dma(st, st);
    __builtin_amdgcn_s_waitcnt(WaitVmLgkm0<(NS - 1) * PER>::value);
    __builtin_amdgcn_s_barrier();
    load(sm, 0, f0);
    for (int kt = 0; kt < nk; kt += NS) {
#pragma unroll
      for (int st = 0; st < NS; ++st) step(st, kt + st);
    }
    __builtin_amdgcn_s_waitcnt(WaitVmLgkm0<0>::value);  // no LDS write may outlive the block
  }

  if (splits > 1) {
    int* dst = part + (int64_t)z * a.T * a.M;
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
    const float ws = mok ? a.wstep[m] : 0.0f;
    const float bs = mok && bias ? from16<BF16>(bias[m]) : 0.0f;
#pragma unroll
    for (int i = 0; i < S::TI; ++i) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int t = t0 + (wt * S::TI + i) * 32 + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
        if (t < a.T && mok) {
          float v = scaled(acc[i][j][e], a.xstep[t], ws);
          if (bias) v = v + bs;
          y[(int64_t)t * a.ldy + m] = to16<BF16>(v);
        }
      }
    }
  }
}

// The sum of the splits' int32 tiles (exact, so their order does not matter), scaled.  Four
// outputs a thread where M allows it.
template <bool BF16, int V>
__global__ __launch_bounds__(256) void k_int8_finish(Int8Args a, int splits,
                                                     const int* __restrict__ part) {
  typedef int ivec __attribute__((ext_vector_type(V)));
  const int64_t n = (int64_t)a.T * a.M;
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V;
  if (i >= n) return;
  const int t = (int)(i / a.M), m = (int)(i - (int64_t)t * a.M);
  ivec s = *(const ivec*)(part + i);
  for (int z = 1; z < splits; ++z) s += *(const ivec*)(part + z * n + i);
  const float xs = a.xstep[t];
  const uint16_t* bias = (const uint16_t*)a.bias;
  uint16_t* y = (uint16_t*)a.y + (int64_t)t * a.ldy + m;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    float v = scaled(s[e], xs, a.wstep[m + e]);
    if (bias) v = v + from16<BF16>(bias[m + e]);
    y[e] = to16<BF16>(v);
  }
}

// ---- few tokens --------------------------------------------------------------------------
//
// Up to 16 tokens the product is bound by reading the weights once.  A block takes 16 RT outputs
// and all tokens; its eight waves take 256-byte pieces of K in turn.  The weights go
// from memory to the operand registers of v_mfma_i32_16x16x64_i8 directly (lane l: 16 bytes of
// row l mod 16 at 16 (l div 16); four instructions cover 256 contiguous bytes of a row), the
// next piece's ahead of the products of this one; the tokens' operands come from L2.  The
// waves' int32 sums are added through LDS.  Result element e of lane l is output 4 (l div 16) + e,
// token l mod 16.  Measured: 16 tokens, 11008 x 4096 15 us (3.0 TB/s), one token, 4096 x 4096 with
// the quantisation 7 to 9 us: short of the memory's rate because a wave has two pieces to load
// between its start and its end.
//
// FUSED (one token): the block first quantises the token into LDS, with the first weights
// already on their way; every block repeats that (a few thousand values from L2) in place of a
// launch before this one.
constexpr int kFewWaves = 8;
constexpr int kFusedChunks = 4;  // 8-column chunks of the token a thread keeps
constexpr int kFusedMaxK = 8 * 64 * kFewWaves * kFusedChunks;

struct FewArgs {
  Int8Args g;
  const void* x16;  // FUSED: the token, its scales and columns
  const float* s;
  int cols;
};

template <int RT, bool FUSED, bool BF16, bool VEC>
__global__ __launch_bounds__(64 * kFewWaves) void k_int8_few(FewArgs f) {
  const Int8Args& a = f.g;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, q = lane >> 4;
  const unsigned first = block_number() * 16u * RT;  // below 2^32 past M, too
  if (first >= (unsigned)a.M) return;                // the whole block
  const int m0 = (int)first;
  const int nch = (a.K + 255) >> 8;

  // rows past the last repeat it and are dropped; pieces past K read the row's start and count 0
  const int8_t* wrow[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) wrow[r] = a.w + (int64_t)min(m0 + 16 * r + lr, a.M - 1) * a.ldw;
  auto load_w = [&](int32x4 (&o)[RT][4], int ch) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = ch * 256 + u * 64 + 16 * q;
      const bool in = k < a.K;
#pragma unroll
      for (int r = 0; r < RT; ++r) o[r][u] = *(const int32x4*)(wrow[r] + (in ? k : 0));
    }
  };
  int32x4 w0[RT][4], w1[RT][4];
  if (wave < nch) load_w(w0, wave);

  float fused_step = 0.0f;
  if constexpr (FUSED) {
    __shared__ uint32_t red[kFewWaves];
    const int n8 = a.K >> 3;  // 8-column chunks (K whole 16-byte pieces)
    float v[kFusedChunks][8];
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < kFusedChunks; ++c) {
      const int ch = tid + c * 64 * kFewWaves;
      if (ch < n8) {
        load_row8<BF16, VEC>((const uint16_t*)f.x16, f.s, f.s ? kFoldDivide : kFoldNone, 8 * ch, f.cols, v[c]);
        top = max_abs8(v[c], top);
      }
    }
    const RowStep st = row_step(block_max<kFewWaves>(top, red));
    fused_step = st.step;
#pragma unroll
    for (int c = 0; c < kFusedChunks; ++c) {
      const int ch = tid + c * 64 * kFewWaves;
      if (ch < n8) *(uint2*)(lds + 8 * ch) = row_codes8(v[c], st);
    }
    __syncthreads();
  }

  // columns past the last token repeat it and are dropped
  const int8_t* xrow = FUSED ? nullptr : a.x + (int64_t)min(lr, a.T - 1) * a.ldx;
  int32x4 acc[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) acc[r] = int32x4{0, 0, 0, 0};
  auto load_x = [&](int32x4 (&x)[4], int ch) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = ch * 256 + u * 64 + 16 * q;
      const int at = k < a.K ? k : 0;
      if constexpr (FUSED) x[u] = *(const int32x4*)(lds + at);
      else x[u] = *(const int32x4*)(xrow + at);
    }
  };
  auto piece = [&](int32x4 (&w)[RT][4], int32x4 (&x)[4], int ch) {
    if (ch == nch - 1) {  // pieces past K count nothing
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int r = 0; r < RT; ++r)
          if (ch * 256 + u * 64 + 16 * q >= a.K) w[r][u] = int32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int r = 0; r < RT; ++r)
        acc[r] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[r][u], x[u], acc[r], 0, 0, 0);
  };
  // a piece's tokens are asked for before the next piece's weights: loads return in order, so
  // waiting for the tokens does not wait for those weights
  for (int ch = wave; ch < nch; ch += 2 * kFewWaves) {
    int32x4 x[4];
    load_x(x, ch);
    if (ch + kFewWaves < nch) load_w(w1, ch + kFewWaves);
    __builtin_amdgcn_sched_barrier(0);
    piece(w0, x, ch);
    if (ch + kFewWaves >= nch) break;
    load_x(x, ch + kFewWaves);
    if (ch + 2 * kFewWaves < nch) load_w(w0, ch + 2 * kFewWaves);
    __builtin_amdgcn_sched_barrier(0);
    piece(w1, x, ch + kFewWaves);
  }

  // the waves' sums, then one (tile, lane) a thread
  __shared__ int32x4 sum[kFewWaves][RT][64];
#pragma unroll
  for (int r = 0; r < RT; ++r) sum[wave][r][lane] = acc[r];
  __syncthreads();
  const uint16_t* bias = (const uint16_t*)a.bias;
  for (int i = tid; i < RT * 64; i += 64 * kFewWaves) {
    const int tile = i >> 6, l = i & 63;
    int32x4 v = sum[0][tile][l];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) v += sum[w][tile][l];
    const int t = l & 15, m = m0 + 16 * tile + 4 * (l >> 4);
    if (t >= a.T) continue;
    const float xs = FUSED ? fused_step : a.xstep[t];
    uint16_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (m + e < a.M) {
        float y = scaled(v[e], xs, a.wstep[m + e]);
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
hipError_t launch_tiles(const Int8Args& a, int splits, int* part, hipStream_t stream) {
  const int tt = (a.T + S::BT - 1) / S::BT, tm = (a.M + S::BM - 1) / S::BM;
  const int64_t tiles = (int64_t)tt * tm;
  if (tiles > kMaxBlocks) return hipErrorInvalidValue;
  dim3 grid = grid_of(tiles);
  grid.z = (unsigned)splits;
  hipLaunchKernelGGL((k_int8_tiles<S, BF16>), grid,
                     dim3(S::THREADS), 0, stream, a, tt, tm, splits, part);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits <= 1) return e;
  const int64_t n = (int64_t)a.T * a.M;
  if (a.M % 4 == 0)
    hipLaunchKernelGGL((k_int8_finish<BF16, 4>), dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0,
                       stream, a, splits, part);
  else
    hipLaunchKernelGGL((k_int8_finish<BF16, 1>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0,
                       stream, a, splits, part);
  return hipGetLastError();
}

template <int RT, bool FUSED, bool VEC>
hipError_t launch_few(const FewArgs& f, hipStream_t stream) {
  const dim3 grid = grid_of((f.g.M + 16 * RT - 1) / (16 * RT)), block(64 * kFewWaves);
  const size_t lds = FUSED ? (size_t)f.g.K : 0;
  if (f.g.bf16)
    hipLaunchKernelGGL((k_int8_few<RT, FUSED, true, VEC>), grid, block, lds, stream, f);
  else
    hipLaunchKernelGGL((k_int8_few<RT, FUSED, false, VEC>), grid, block, lds, stream, f);
  return hipGetLastError();
}

template <bool BF16>
hipError_t launch_plan(const Int8Args& a, const Int8Plan& p, int* part, hipStream_t stream) {
  switch (p.form) {
    case kTile32: return launch_tiles<Tile<32, 128, 1, 4, 4>, BF16>(a, p.splits, part, stream);
    case kTile64: return launch_tiles<Tile<64, 128, 2, 2, 3>, BF16>(a, p.splits, part, stream);
    case kTile128: return launch_tiles<Tile<128, 128, 2, 2, 2>, BF16>(a, p.splits, part, stream);
    default: return launch_tiles<Tile<256, 256, 2, 8, 2>, BF16>(a, 1, nullptr, stream);
  }
}

}  // namespace

size_t int8_matmul_workspace(int64_t T, int64_t M, int64_t K) {
  const Int8Plan p = int8_plan(T, M, K);
  return p.splits > 1 ? (size_t)p.splits * T * M * sizeof(int) : 0;
}

hipError_t launch_int8_matmul(const Int8Args& a, void* workspace, hipStream_t stream) {
  if (a.T <= 0 || a.M <= 0) return hipSuccess;
  const Int8Plan p = int8_plan(a.T, a.M, a.K);
  if (p.form < kTile32) {
    const FewArgs f{a, nullptr, nullptr, 0};
    return few_rows(a.M) == 2 ? launch_few<2, false, false>(f, stream) : launch_few<1, false, false>(f, stream);
  }
  return a.bf16 ? launch_plan<true>(a, p, (int*)workspace, stream)
                : launch_plan<false>(a, p, (int*)workspace, stream);
}

bool int8_linear_fused(int64_t T, int64_t K) { return T == 1 && K <= kFusedMaxK; }

hipError_t launch_int8_linear_fused(const Int8Args& a, const void* x, const float* s, int cols,
                                    hipStream_t stream) {
  if (a.T <= 0 || a.M <= 0) return hipSuccess;
  const FewArgs f{a, x, s, cols};
  const bool vec = row_vector_loads(x, 0, s);
  const bool two = few_rows(a.M) == 2;
  if (vec) return two ? launch_few<2, true, true>(f, stream) : launch_few<1, true, true>(f, stream);
  return two ? launch_few<2, true, false>(f, stream) : launch_few<1, true, false>(f, stream);
}

}  // namespace awq
