// Product in 8-bit integers: y[t][m] = float(sum_i x[t][i] w[m][i]) xstep[t] wstep[m] + bias[m].
//
// Pages: "AWQ" scholia-log notes §2.3 (symmetric integer quantiser); the product is exact in
// int32, so neither the order of the sum nor a split of it changes a result.
//
// Tiles (many tokens): both operands are K-contiguous bytes.  A block computes BT tokens x BM
// outputs from tiles of 128 bytes of K, which move global -> LDS by DMA into a ring of two
// stages (rows of 128 bytes, the 16-byte chunk index XOR-swizzled with the row, so that the
// fragment reads of 32 rows are free of bank conflicts), and feeds
// v_mfma_i32_32x32x32_i8: lane l supplies 16 bytes of row l mod 32 at chunk 2 k + l div 32 for
// both operands; element e of the result is row 8 (e div 4) + 4 (l div 32) + e mod 4 of the
// first operand (token), column l mod 32 of the second (output).  Rows past the matrices and
// chunks past K lie outside the buffer resources or take an out-of-range offset and arrive as
// zeros.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "int8_quant.h"
#include "mfma_dma.h"
#include "serve_internal.h"

namespace awq {

namespace {

// y = (float(acc) xstep) wstep + bias, each operation rounded once in fp32, then to 16 bits.
__device__ __forceinline__ float scaled(int acc, float xs, float ws) {
  return (float)acc * xs * ws;
}

template <int BT_, int BM_, int WT_, int WM_>
struct Tile {
  static constexpr int BT = BT_, BM = BM_, WT = WT_, WM = WM_;
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

template <class S, bool BF16>
__global__ __launch_bounds__(S::THREADS) void k_int8_tiles(Int8Args a, int tiles_t, int tiles_m) {
  __shared__ __attribute__((aligned(1024))) uint8_t sm0[S::BYTES];
  __shared__ __attribute__((aligned(1024))) uint8_t sm1[S::BYTES];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63;
  const int wt = wave / S::WM, wm = wave % S::WM;

  // Blocks go to the 8 XCDs in turn; renumbered so that each XCD walks a contiguous range of
  // tiles in bands of 8 token tiles, whose panels its compute units share in that XCD's L2.
  constexpr int kBand = 8;
  const int total = tiles_t * tiles_m;
  const int b = blockIdx.x, xcd = b & 7, local = b >> 3;
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
  const unsigned ldsb[2] = {lds_address(sm0), lds_address(sm1)};
  const int nk = (a.K + 2 * S::BK - 1) / (2 * S::BK) * 2;  // whole pairs of stages

  auto dma = [&](int st, int kt) {
    const int k0 = kt * S::BK;
    const bool oke = k0 + ce * 16 < a.K, oko = k0 + co * 16 < a.K;
#pragma unroll
    for (int j = 0; j < S::DMA_X; ++j) {
      const bool odd = (wave * S::DMA_X + j) & 1;
      const unsigned r = row_x + 8 * j;
      const unsigned v = (odd ? oko : oke) && r < (unsigned)rows_x
                             ? r * ldx + (odd ? co : ce) * 16 : kOut;
      lds_dma16(rx, ldsb[st] + (wave * S::DMA_X + j) * 1024u, v, k0);
    }
#pragma unroll
    for (int j = 0; j < S::DMA_W; ++j) {
      const bool odd = (wave * S::DMA_W + j) & 1;
      const unsigned r = row_w + 8 * j;
      const unsigned v = (odd ? oko : oke) && r < (unsigned)rows_w
                             ? r * ldw + (odd ? co : ce) * 16 : kOut;
      lds_dma16(rw, ldsb[st] + S::X_BYTES + (wave * S::DMA_W + j) * 1024u, v, k0);
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

  // Two stages in flight; a stage is refilled after the barrier that follows its last
  // fragment read, and the DMAs past the end of K read zeros into a slot nobody uses, so the
  // number in flight, hence the vmcnt to wait for, is constant.
  Frag f0, f1;
  auto step = [&](const uint8_t* cur, const uint8_t* next, int st, int kt) {
#pragma unroll
    for (int ks = 0; ks + 2 < S::KSTEPS; ks += 2) {
      load(cur, ks + 1, f1);
      mma(f0);
      load(cur, ks + 2, f0);
      mma(f1);
    }
    load(cur, S::KSTEPS - 1, f1);
    mma(f0);
    __builtin_amdgcn_s_waitcnt(WaitVmLgkm0<0>::value);  // stage kt + 1 has landed
    __builtin_amdgcn_s_barrier();
    dma(st, kt + 2);
    load(next, 0, f0);
    mma(f1);
  };
  if (nk > 0) {
    dma(0, 0);
    dma(1, 1);
    __builtin_amdgcn_s_waitcnt(WaitVmLgkm0<S::DMA_X + S::DMA_W>::value);
    __builtin_amdgcn_s_barrier();
    load(sm0, 0, f0);
    for (int kt = 0; kt < nk; kt += 2) {
      step(sm0, sm1, 0, kt);
      step(sm1, sm0, 1, kt + 1);
    }
    __builtin_amdgcn_s_waitcnt(WaitVmLgkm0<0>::value);  // no LDS write may outlive the block
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

template <class S, bool BF16>
hipError_t launch_tiles(const Int8Args& a, hipStream_t stream) {
  const int tt = (a.T + S::BT - 1) / S::BT, tm = (a.M + S::BM - 1) / S::BM;
  if ((long long)tt * tm > 0x7fffffffLL) return hipErrorInvalidValue;
  hipLaunchKernelGGL((k_int8_tiles<S, BF16>), dim3((unsigned)(tt * tm)), dim3(S::THREADS), 0,
                     stream, a, tt, tm);
  return hipGetLastError();
}

}  // namespace

size_t int8_matmul_workspace(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_int8_matmul(const Int8Args& a, void*, hipStream_t stream) {
  if (a.T <= 0 || a.M <= 0) return hipSuccess;
  using S = Tile<128, 128, 2, 2>;
  return a.bf16 ? launch_tiles<S, true>(a, stream) : launch_tiles<S, false>(a, stream);
}

}  // namespace awq
