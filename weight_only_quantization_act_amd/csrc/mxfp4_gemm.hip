// Product in MXFP4: y[t][m] = sum_i x[t][i] w[m][i] + bias[m], both operands blocks of 32 4-bit
// floating-point elements with a power of two each.
//
// Pages: "AWQ" scholia-log notes §1.1 (the layer's product); "AWQ量化技术解析" (kwkr.cn) §4.2
// (dequantisation fused into the product): here the matrix cores take the codes and the scales as
// they are.  An instruction adds 64 or 128 products of 4-bit elements (exact, multiples of 1/4 times a
// power of two) to the running fp32 sum, within 2^-22 of its largest term or result (measured); subnormals
// are kept.
//
// Tiles: a block computes BT tokens x BM outputs from stages of 128 bytes of K (256 columns) that
// move global -> LDS by DMA into a ring of NS (rows of 128 bytes, the 16-byte chunk index XOR-swizzled
// with the row).  v_mfma_scale_f32_32x32x64_f8f6f4 takes, in lane l, one block of row l mod 32 of both
// operands and its scale byte.  Which columns an instruction multiplies is free as long as both
// operands agree: step k of a stage takes block 4 (l div 32) + k, so that a lane's four scales of a
// stage are one 32-bit word of the scales' layout, byte k of it chosen by the instruction.  The
// words of a tile's rows are contiguous ([column word][row]) and come by DMA as well.  Element e of the
// result is row 8 (e div 4) + 4 (l div 32) + e mod 4 of the first operand (output), column l mod 32 of
// the second (token).  Rows past the matrices and chunks past K arrive as zeros, or as scales of rows
// that are dropped.
//
// Large products run at the power limit: 8192 tokens of 28672 x 8192 939-962 us, 4.0-4.1 PFLOP/s (matrix
// cores busy 54% of the cycles at 1.81 GHz; the same instructions alone on the same data 6.2 PFLOP/s; without
// the refills the loop takes 16% less, without its LDS reads 10%, without waiting for the refills nothing).
// Not faster, in us on 859 of the kernel alone: four waves of 128 x 128 with a third fewer LDS reads 910,
// operand reads placed between the products by hand 885, the loop over one stage with its slot in a
// register 851 (128 x 128 tiles 22.2 for 21.3), bands of 4, 6 and 16 tiles 855, 856, 866, stages of 64
// bytes, instructions of 16 x 16 x 128.  Products with a tile or two a compute unit are bound by each step's
// chain of barrier, products, reads and refills (333 tokens of 5120 x 13824 21.2-22.2 us, 2.1-2.2 PFLOP/s, 0.35
// us a step; matrix cores busy 17%; the refills alone would take 0.24; weights that no cache holds 27.7): neither
// fewer LDS reads, deeper rings nor two stages a barrier shorten it.
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

template <int BT_, int BM_, int WT_, int WM_, int KG_, int NS_, bool WHOLE_>
struct MxTile {
  static constexpr int BT = BT_, BM = BM_, WT = WT_, WM = WM_;
  static constexpr int KG = KG_, NS = NS_;  // groups of waves, which take the steps in turn, stages of each
  static constexpr bool WHOLE = WHOLE_;     // a stage's operands are read one stage ahead (else an instruction)
  static constexpr int BK = 128;            // bytes of K a stage
  static constexpr int WAVES = WT * WM, THREADS = 64 * WAVES * KG;
  static constexpr int TI = BT / WT / 32, MI = BM / WM / 32;
  static constexpr int X_BYTES = BT * BK, CODES = (BT + BM) * BK;
  static constexpr int XS_BYTES = 2 * 4 * BT, BYTES = CODES + 2 * 4 * (BT + BM);
  static constexpr int DMA_X = X_BYTES / 1024 / WAVES, DMA_W = BM * BK / 1024 / WAVES;
  // scales: DMAs of 64 words; where they do not divide evenly a wave repeats another's
  static constexpr int S_X = 2 * BT / 64, S_ALL = 2 * (BT + BM) / 64;
  static constexpr int DMA_S = (S_ALL + WAVES - 1) / WAVES;
  static constexpr int PER = DMA_X + DMA_W + DMA_S;
  static_assert(X_BYTES % (1024 * WAVES) == 0 && BM * BK % (1024 * WAVES) == 0 && S_X >= 1,
                "each wave loads a part of both operands");
  static_assert(TI >= 1 && MI >= 1, "each wave has a 32 x 32 tile at least");
  // Physical chunk of a row's chunk c: c ^ swz(row).  Eight consecutive rows' chunks c fall on eight
  // different 16-byte groups of banks.
  __device__ static int swz(int row) { return (row & 7) ^ ((row >> 3) & 1); }
  // After the last step LDS holds the sums of the groups but the first, then the tile's results in rows
  // 16 bytes apart more than their length (bank conflicts), then the biases.
  static constexpr int OUT = BM * 2 + 16;
  static constexpr int RESULTS = (KG - 1) * BT * BM * 4;
  static constexpr int BIAS = RESULTS + BT * OUT;
  static constexpr int LDS = KG * NS * BYTES > BIAS + 4 * BM ? KG * NS * BYTES : BIAS + 4 * BM;
};

template <class S, bool BF16>
__global__ __launch_bounds__(S::THREADS) void k_mxfp4_tiles(MxArgs a, int tiles_t, int tiles_m) {
  constexpr int NS = S::NS;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::LDS];
  const int tid = threadIdx.x;
  const int all = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int group = all / S::WAVES, wave = all % S::WAVES;
  const int lane = tid & 63;
  uint8_t* const sm = lds + group * NS * S::BYTES;
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

  // steps of 128 bytes, which the groups take in turn, each the same number
  const int steps = (a.KB + S::BK - 1) / S::BK;
  const int n_steps = (steps + S::KG - 1) / S::KG;
  const int words = (a.KB + 63) >> 6;  // scale words a row

  // A wave-DMA fills 8 rows of 128 bytes: lane l its row l / 8, physical chunk l % 8, which
  // holds logical chunk (l % 8) ^ swz(row).  swz depends on row mod 16, so on the parity of
  // the 8-row block as well as on the lane.  Rows past the last lie out of range.
  constexpr unsigned kOut = 0x80000000u;
  const int dr = lane >> 3;
  const int ce = (lane & 7) ^ S::swz(dr), co = (lane & 7) ^ S::swz(dr + 8);
  const unsigned ldsb = lds_address(sm);
  unsigned vx[S::DMA_X], vw[S::DMA_W];
#pragma unroll
  for (int j = 0; j < S::DMA_X; ++j) {
    const int p = wave * S::DMA_X + j, r = 8 * p + dr;
    vx[j] = r < rows_x ? (unsigned)r * ldx + (p & 1 ? co : ce) * 16 : kOut;
  }
#pragma unroll
  for (int j = 0; j < S::DMA_W; ++j) {
    const int p = wave * S::DMA_W + j, r = 8 * p + dr;
    vw[j] = r < rows_w ? (unsigned)r * ldw + (p & 1 ? co : ce) * 16 : kOut;
  }
  // Scales: the step's two words of the tile's rows, [2][BT], then [2][BM].  The address walks with
  // the steps; a lane's offset in the rows of words stays.
  const uint32_t* sp[S::DMA_S];
  unsigned vs[S::DMA_S];
  bool sq[S::DMA_S];  // the lane's word is the second one
#pragma unroll
  for (int j = 0; j < S::DMA_S; ++j) {
    const int d = (wave * S::DMA_S + j) % S::S_ALL;
    const bool is_x = d < S::S_X;
    const int64_t ld = is_x ? a.ldxs : a.ldws;
    const int i = (is_x ? d : d - S::S_X) * 64 + lane, n = is_x ? S::BT : S::BM;
    const int q = i / n, r = i % n;
    sp[j] = (is_x ? a.xs + t0 : a.ws + m0) + 2 * (int64_t)group * ld;
    vs[j] = r < (is_x ? rows_x : rows_w) ? ((unsigned)q * (unsigned)ld + r) * 4u : kOut;
    sq[j] = q == 1;
  }

  // Piece j of a wave's part of its group's step kt (called with kt = 0, 1, 2, ...).
  auto dma_piece = [&](int st, int kt, int j) {
    const int at = kt * S::KG + group, k0 = at * S::BK;
    const bool in = at < steps;
    if (j < S::DMA_X + S::DMA_W) {
      const bool is_x = j < S::DMA_X;
      const int i = is_x ? j : j - S::DMA_X;
      const int p = wave * (is_x ? S::DMA_X : S::DMA_W) + i;
      const bool ok = in && k0 + (p & 1 ? co : ce) * 16 < a.KB;
      lds_dma16(is_x ? rx : rw, ldsb + st * S::BYTES + (is_x ? 0 : S::X_BYTES) + p * 1024u,
                ok ? (is_x ? vx[i] : vw[i]) : kOut, k0);
    } else {
      const int i = j - S::DMA_X - S::DMA_W;
      const int d = (wave * S::DMA_S + i) % S::S_ALL;
      const int nq = in ? words - 2 * at : 0;
      lds_dma4(buffer_rsrc(sp[i], kOut), ldsb + st * S::BYTES + S::CODES + d * 256u,
               nq > (sq[i] ? 1 : 0) ? vs[i] : kOut);
      sp[i] += 2 * S::KG * (d < S::S_X ? a.ldxs : a.ldws);
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
  // The bytes of the last step's words behind the row's last block may be any, 255 (NaN) among them.
  const int left = (a.KB >> 4) - 8 * ((n_steps - 1) * S::KG + group) - 4 * fh;  // the lane's blocks of that step
  const int kept = left >= 4 ? -1 : left > 0 ? (1 << (8 * left)) - 1 : 0;
  auto clear_behind = [&](Scales& s) {
#pragma unroll
    for (int i = 0; i < S::TI; ++i) s.x[i] &= kept;
#pragma unroll
    for (int i = 0; i < S::MI; ++i) s.w[i] &= kept;
  };
  floatx16 acc[S::TI][S::MI];
#pragma unroll
  for (int i = 0; i < S::TI; ++i)
#pragma unroll
    for (int j = 0; j < S::MI; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  // outputs are the rows of the result, tokens its columns
  auto mma1 = [&](auto ks, int i, int j, const Frag& f, const Scales& s) {
    constexpr int B = decltype(ks)::value;
    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
        operand(f.w[j]), operand(f.x[i]), acc[i][j], kFp4, kFp4, B, s.w[j], B, s.x[i]);
  };
  auto mma = [&](auto ks, const Frag& f, const Scales& s) {
#pragma unroll
    for (int i = 0; i < S::TI; ++i)
#pragma unroll
      for (int j = 0; j < S::MI; ++j) mma1(ks, i, j, f, s);
  };
  using std::integral_constant;

  // NS stages in flight; a stage is refilled after the barrier that follows its last fragment
  // read, and the DMAs past the end of K read zeros into a slot nobody uses, so the number in
  // flight, hence the vmcnt to wait for, is constant.
  auto begin = [&] {
#pragma unroll
    for (int st = 0; st < NS; ++st)
#pragma unroll
      for (int j = 0; j < S::PER; ++j) dma_piece(st, st, j);
    __builtin_amdgcn_s_waitcnt(WaitVmLgkm0<(NS - 1) * S::PER>::value);
    if constexpr (S::WAVES > 1) __builtin_amdgcn_s_barrier();
  };
  auto landed = [&] {  // the step after this one's
    __builtin_amdgcn_s_waitcnt(WaitVmLgkm0<(NS - 2) * S::PER>::value);
    if constexpr (S::WAVES > 1) __builtin_amdgcn_s_barrier();
  };
  if (n_steps == 0) {
  } else if constexpr (S::WHOLE) {
    // One or two tiles a wave: a step has too few products to hide its own reads, so a whole stage's
    // operands are read during the products of the one before (50 tokens of 11008 x 4096 on 64 x 64
    // 7.8 -> 7.2 us; 512 of 5120 x 13824 on 128 x 128 in three stages, one block a unit, 43.5 -> 29.2).
    Frag f[2][4];
    Scales s[2];
    auto read = [&](int st, Frag (&to)[4], Scales& ts) {
      load_scales(sm + st * S::BYTES, ts);
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) load(sm + st * S::BYTES, ks, to[ks]);
    };
    begin();
    read(0, f[0], s[0]);
    constexpr int U = NS % 2 ? 2 * NS : NS;
    for (int kt = 0; kt < n_steps - 1; kt += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (kt + u >= n_steps - 1) break;
        landed();
        const uint8_t* next = sm + (u + 1) % NS * S::BYTES;
        // Products first, a part of the next stage's reads and of the refill behind each: a refill's instruction
        // waits for the others' addresses, and a wave that issues them all first leaves the matrix
        // cores idle meanwhile (333 tokens of 5120 x 13824 25.0 -> 22.9 us on the device alone).
        auto part = [&](auto ks) {
          mma(ks, f[u & 1][decltype(ks)::value], s[u & 1]);
          __builtin_amdgcn_sched_barrier(0);
          load(next, decltype(ks)::value, f[~u & 1][decltype(ks)::value]);
#pragma unroll
          for (int j = decltype(ks)::value * S::PER / 4; j < (decltype(ks)::value + 1) * S::PER / 4; ++j)
            dma_piece(u % NS, kt + u + NS, j);
          __builtin_amdgcn_sched_barrier(0);
        };
        __builtin_amdgcn_sched_barrier(0);
        load_scales(next, s[~u & 1]);
        part(integral_constant<int, 0>{});
        part(integral_constant<int, 1>{});
        part(integral_constant<int, 2>{});
        part(integral_constant<int, 3>{});
      }
    }
    auto last = [&](const Frag (&of)[4], Scales& os) {  // its operands are here, nothing is refilled
      clear_behind(os);
      mma(integral_constant<int, 0>{}, of[0], os);
      mma(integral_constant<int, 1>{}, of[1], os);
      mma(integral_constant<int, 2>{}, of[2], os);
      mma(integral_constant<int, 3>{}, of[3], os);
    };
    if (n_steps & 1) last(f[0], s[0]);  // (U is even)
    else last(f[1], s[1]);
  } else {
    Frag f0, f1;
    Scales sc, sn;
    begin();
    load_scales(sm, sc);
    load(sm, 0, f0);
    // a step's products but its last instruction's
    auto most = [&](const uint8_t* cur) {
      load(cur, 1, f1);
      mma(integral_constant<int, 0>{}, f0, sc);
      load(cur, 2, f0);
      mma(integral_constant<int, 1>{}, f1, sc);
      load(cur, 3, f1);
      mma(integral_constant<int, 2>{}, f0, sc);
    };
    for (int kt = 0; kt < n_steps - 1; kt += NS) {
#pragma unroll
      for (int st = 0; st < NS; ++st) {
        if (kt + st >= n_steps - 1) break;
        const uint8_t* next = sm + (st + 1) % NS * S::BYTES;
        most(sm + st * S::BYTES);
        landed();
        load_scales(next, sn);
        load(next, 0, f0);
        // the refill's instructions between the products, which keep the matrix cores busy meanwhile
        constexpr int N = S::TI * S::MI;
#pragma unroll
        for (int n = 0; n < N; ++n) {
          mma1(integral_constant<int, 3>{}, n / S::MI, n % S::MI, f1, sc);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int p = n * S::PER / N; p < (n + 1) * S::PER / N; ++p) dma_piece(st, kt + st + NS, p);
          __builtin_amdgcn_sched_barrier(0);
        }
        sc = sn;
      }
    }
    clear_behind(sc);  // the last step, without a refill
    most(sm + (n_steps - 1) % NS * S::BYTES);
    mma(integral_constant<int, 3>{}, f1, sc);
  }
  __builtin_amdgcn_s_waitcnt(WaitVmLgkm0<0>::value);  // no LDS write may come after this
  __syncthreads();

  if constexpr (S::KG > 1) {  // the groups' sums, added in their order
    floatx4* const sums = (floatx4*)lds;
    auto slot = [&](int g, int i, int j, int e) {
      return (((g - 1) * S::WAVES + wave) * S::TI * S::MI * 4 + (i * S::MI + j) * 4 + e) * 64 + lane;
    };
    if (group > 0) {
#pragma unroll
      for (int i = 0; i < S::TI; ++i)
#pragma unroll
        for (int j = 0; j < S::MI; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sums[slot(group, i, j, e)] = floatx4{acc[i][j][4 * e], acc[i][j][4 * e + 1], acc[i][j][4 * e + 2], acc[i][j][4 * e + 3]};
    }
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (int g = 1; g < S::KG; ++g)
#pragma unroll
        for (int i = 0; i < S::TI; ++i)
#pragma unroll
          for (int j = 0; j < S::MI; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const floatx4 v = sums[slot(g, i, j, e)];
#pragma unroll
              for (int k = 0; k < 4; ++k) acc[i][j][4 * e + k] += v[k];
            }
    }
  }

  // Results through LDS, so that stores fill whole lines: a lane has four consecutive outputs of a
  // token at a time; the rows of the tile are then read 16 bytes a lane (8192 tokens of 28672 x 8192
  // 945 -> 889 us).
  uint8_t* const results = lds + S::RESULTS;
  const uint16_t* bias = (const uint16_t*)a.bias;
  float* const lbias = (float*)(lds + S::BIAS);
  if (bias) {
    for (int m = tid; m < S::BM; m += S::THREADS) lbias[m] = m < rows_w ? from16<BF16>(bias[m0 + m]) : 0.0f;
    __syncthreads();
  }
  if (group == 0) {
#pragma unroll
    for (int i = 0; i < S::TI; ++i)
#pragma unroll
      for (int j = 0; j < S::MI; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int t = (wt * S::TI + i) * 32 + fr;
          const int m = (wm * S::MI + j) * 32 + 8 * g + 4 * fh;
          floatx4 o = {acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
          if (bias) {
            const floatx4 bb = *(const floatx4*)(lbias + m);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = o[k] + bb[k];
          }
          uint2 p;
          p.x = to16<BF16>(o[0]) | ((uint32_t)to16<BF16>(o[1]) << 16);
          p.y = to16<BF16>(o[2]) | ((uint32_t)to16<BF16>(o[3]) << 16);
          *(uint2*)(results + t * S::OUT + 2 * m) = p;
        }
  }
  __syncthreads();
  uint16_t* y = (uint16_t*)a.y + (int64_t)t0 * a.ldy + m0;
  auto store = [&](auto stream) {
    constexpr int kPer = S::BM / 8;
    for (int c = tid; c < S::BT * kPer; c += S::THREADS) {
      const int t = c / kPer, m = 8 * (c % kPer);
      if (t >= rows_x || m >= rows_w) continue;
      const u32x4 v = *(const u32x4*)(results + t * S::OUT + 2 * m);
      uint16_t* o = y + (int64_t)t * a.ldy + m;
      if (m + 8 <= rows_w) {  // (16 bytes at any even address)
        if constexpr (decltype(stream)::value) __builtin_nontemporal_store(v, (u32x4_at2*)o);
        else *(u32x4_at2*)o = v;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (m + e < rows_w) o[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
      }
    }
  };
  // Results that no cache will hold are kept from pushing the panels out of it: output of 470 MB 882
  // -> 843 us, of 90 MB 97 -> 99 us.
  if ((int64_t)a.T * a.M * 2 > kCacheBytes) store(std::true_type{});
  else store(std::false_type{});
}

// ---- few tokens --------------------------------------------------------------------------
//
// A few tokens' product is bound by reading the weights once.  A block takes 16 outputs
// and all tokens, TT tiles of 16; its eight waves take 256-byte pieces of K (512 columns) in turn.  The weights go
// from memory to the operand registers of v_mfma_scale_f32_16x16x128_f8f6f4 directly: lane l has
// row l mod 16 and the 64 bytes from 64 (l div 16) of a piece, whose four blocks' scales are one word;
// instruction u takes block u of each lane.  The next piece's loads are ahead of the products of
// this one; the tokens' operands come from L2.  The waves' fp32 sums are added through LDS in their
// order.  Result element e of lane l is output 4 (l div 16) + e, token l mod 16.
//
// One token through 4096 x 4096 with its quantisation and scales 5.4 us, without scales 5.0 (9 MB: 1.9 TB/s with
// start and end of the launch), the product alone 4.6, of 16 tokens 5.3, of 17 5.6; 1.2 less where the
// weights are in the last-level cache.
//
// FUSED > 0: the block first quantises the tokens into LDS, a lane 8 columns of so many tokens together, with
// the first weights already on their way; every block repeats that (a few thousand values from L2) in place of
// a launch before this one.
constexpr int kFewWaves = 8;

struct MxFewArgs {
  MxArgs g;
  const uint16_t* x16;  // FUSED > 0: the tokens, their scales, columns and row stride
  const float* s;
  int64_t ldx16;
  int cols;
};

template <int FUSED, int TT, bool BF16>
__global__ __launch_bounds__(64 * kFewWaves) void k_mxfp4_few(MxFewArgs f) {
  const MxArgs& a = f.g;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];  // FUSED > 0: codes [T][pieces 256], words [T][4 pieces]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, q = lane >> 4;
  const unsigned first = block_number() * 16u;  // below 2^32 past M, too
  if (first >= (unsigned)a.M) return;           // the whole block
  const int m0 = (int)first;
  const int nch = (a.KB + 255) >> 8;
  const int words = (a.KB + 63) >> 6;

  // rows past the last repeat it and are dropped; blocks past K read the row's start and count 0
  struct Piece {
    int32x4 v[4];
    int s;
  };
  const int row = min(m0 + lr, a.M - 1);
  const uint8_t* const wrow = a.w + (int64_t)row * a.ldw;
  const uint32_t* const srow = a.ws + row;
  auto load_w = [&](Piece& o, int ch) {
    const int k = ch * 256 + 64 * q, word = 4 * ch + q;
    o.s = (int)srow[(int64_t)(word < words ? word : 0) * a.ldws];
#pragma unroll
    for (int u = 0; u < 4; ++u) o.v[u] = *(const int32x4*)(wrow + (k + 16 * u < a.KB ? k + 16 * u : 0));
  };
  Piece p0, p1;
  if (wave < nch) load_w(p0, wave);

  uint32_t* const lwords = (uint32_t*)(lds + (size_t)a.T * nch * 256);
  if constexpr (FUSED > 0) {
    const int n8 = nch * 64;  // 8-column chunks of whole pieces
    const int T = FUSED == 1 ? 1 : a.T;
    for (int i = tid; i < (T + FUSED - 1) / FUSED * n8; i += 64 * kFewWaves) {
      // sixteen lanes have the same tokens and one word
      const int t0 = FUSED == 1 ? 0 : i / n8 * FUSED, ch = FUSED == 1 ? i : i % n8;
      u32x4 raw[FUSED];
#pragma unroll
      for (int k = 0; k < FUSED; ++k) raw[k] = raw8(f.x16 + min(t0 + k, T - 1) * f.ldx16, 8 * ch, f.cols);
      float sv[8];
      double inv[8];
      if (f.s) {
        floats8(f.s, 8 * ch, f.cols, 1.0f, sv);
        if constexpr (FUSED > 1) {
#pragma unroll
          for (int j = 0; j < 8; ++j) inv[j] = reciprocal(sv[j]);
        }
      }
#pragma unroll
      for (int k = 0; k < FUSED; ++k) {
        const int t = t0 + k;
        if (t >= T) break;  // sixteen lanes together
        float v[8];
        values8<BF16>(raw[k], v);
        if (f.s) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = FUSED > 1 ? (float)((double)v[j] * inv[j]) : v[j] / sv[j];
        }
        uint32_t byte;
        const uint32_t c = mx_codes8(v, byte);
        *(uint32_t*)(lds + (size_t)t * nch * 256 + 4 * ch) = c;
        const uint32_t w = mx_scale_word(byte);
        if ((ch & 15) == 0) lwords[t * nch * 4 + (ch >> 4)] = w;
      }
    }
    __syncthreads();
  }

  // columns past the last token repeat it and are dropped
  floatx4 acc[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) acc[i] = floatx4{0.f, 0.f, 0.f, 0.f};
  auto load_x1 = [&](Piece& o, int ch, int tok) {
    const int k = ch * 256 + 64 * q, word = 4 * ch + q;
    if constexpr (FUSED > 0) {
      o.s = (int)lwords[tok * nch * 4 + word];
#pragma unroll
      for (int u = 0; u < 4; ++u) o.v[u] = *(const int32x4*)(lds + (size_t)tok * nch * 256 + k + 16 * u);
    } else {
      o.s = (int)a.xs[(int64_t)(word < words ? word : 0) * a.ldxs + tok];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        o.v[u] = *(const int32x4*)(a.x + (int64_t)tok * a.ldx + (k + 16 * u < a.KB ? k + 16 * u : 0));
    }
  };
  auto load_x = [&](Piece (&o)[TT], int ch) {
#pragma unroll
    for (int i = 0; i < TT; ++i) load_x1(o[i], ch, min(16 * i + lr, a.T - 1));
  };
  auto piece = [&](Piece& w, Piece (&x)[TT], int ch) {
    if (ch == nch - 1) {  // blocks past K count nothing (their scales may be any row's)
      const int k = ch * 256 + 64 * q;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (k + 16 * u >= a.KB) {
          w.v[u] = int32x4{0, 0, 0, 0};
          w.s = w.s & ~(255 << (8 * u));
#pragma unroll
          for (int i = 0; i < TT; ++i) x[i].s = x[i].s & ~(255 << (8 * u));
        }
    }
    auto step = [&](auto uu) {
      constexpr int u = decltype(uu)::value;
#pragma unroll
      for (int i = 0; i < TT; ++i)
        acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(w.v[u]), operand(x[i].v[u]), acc[i], kFp4,
                                                                  kFp4, u, w.s, u, x[i].s);
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
  };
  // a piece's tokens are asked for before the next piece's weights: loads return in order, so
  // waiting for the tokens does not wait for those weights
  for (int ch = wave; ch < nch; ch += 2 * kFewWaves) {
    Piece x[TT];
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

  // the waves' sums, then one lane's four outputs a thread, a tile of tokens a wave
  __shared__ floatx4 sum[TT][kFewWaves][64];
#pragma unroll
  for (int i = 0; i < TT; ++i) sum[i][wave][lane] = acc[i];
  __syncthreads();
  if (wave >= TT) return;
  floatx4 v = sum[wave][0][lane];
#pragma unroll
  for (int w = 1; w < kFewWaves; ++w) {
    const floatx4 o = sum[wave][w][lane];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += o[e];
  }
  const int t = 16 * wave + lr, m = m0 + 4 * q;
  if (t >= a.T) return;
  const uint16_t* bias = (const uint16_t*)a.bias;
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
  if (m + 4 <= a.M) {
    typedef uint32_t u32x2_at2 __attribute__((ext_vector_type(2), aligned(2)));
    *(u32x2_at2*)y = u32x2_at2{o[0] | ((uint32_t)o[1] << 16), o[2] | ((uint32_t)o[3] << 16)};
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (m + e < a.M) y[e] = o[e];
  }
}

template <class S, bool BF16>
hipError_t launch_tiles(const MxArgs& a, hipStream_t stream) {
  const int tt = (a.T + S::BT - 1) / S::BT, tm = (a.M + S::BM - 1) / S::BM;
  const int64_t tiles = (int64_t)tt * tm;
  if (tiles > kMaxBlocks) return hipErrorInvalidValue;
  hipLaunchKernelGGL((k_mxfp4_tiles<S, BF16>), grid_of(tiles), dim3(S::THREADS), 0, stream, a, tt, tm);
  return hipGetLastError();
}

template <int FUSED, int TT>
hipError_t launch_few(const MxFewArgs& f, hipStream_t stream) {
  const dim3 grid = grid_of((f.g.M + 15) / 16), block(64 * kFewWaves);
  const size_t lds = FUSED > 0 ? (size_t)f.g.T * ((f.g.KB + 255) / 256) * (256 + 16) : 0;
  if (f.g.bf16)
    hipLaunchKernelGGL((k_mxfp4_few<FUSED, TT, true>), grid, block, lds, stream, f);
  else
    hipLaunchKernelGGL((k_mxfp4_few<FUSED, TT, false>), grid, block, lds, stream, f);
  return hipGetLastError();
}

template <bool BF16>
hipError_t launch_form(const MxArgs& a, int form, hipStream_t stream) {
  switch (form) {
    case kMxTile32K: return launch_tiles<MxTile<32, 32, 1, 1, 4, 4, true>, BF16>(a, stream);
    case kMxTile32x64K: return launch_tiles<MxTile<32, 64, 1, 2, 2, 3, true>, BF16>(a, stream);
    case kMxTile64K: return launch_tiles<MxTile<64, 64, 2, 2, 2, 3, true>, BF16>(a, stream);
    case kMxTile64: return launch_tiles<MxTile<64, 64, 2, 2, 1, 3, true>, BF16>(a, stream);
    case kMxTile64x128: return launch_tiles<MxTile<64, 128, 2, 4, 1, 3, true>, BF16>(a, stream);
    case kMxTile128W: return launch_tiles<MxTile<128, 128, 4, 2, 1, 3, true>, BF16>(a, stream);
    case kMxTile128: return launch_tiles<MxTile<128, 128, 4, 2, 1, 2, false>, BF16>(a, stream);
    default: return launch_tiles<MxTile<256, 256, 4, 2, 1, 2, false>, BF16>(a, stream);
  }
}

}  // namespace

hipError_t launch_mxfp4_matmul(const MxArgs& a, hipStream_t stream) {
  if (a.T <= 0 || a.M <= 0) return hipSuccess;
  const int form = mxfp4_form(a.T, a.M, a.KB);
  if (form == kMxFew) {
    const MxFewArgs f{a, nullptr, nullptr, 0, 0};
    return a.T <= 16 ? launch_few<0, 1>(f, stream) : launch_few<0, 2>(f, stream);
  }
  return a.bf16 ? launch_form<true>(a, form, stream) : launch_form<false>(a, form, stream);
}

// Where tokens times columns are few.  Fused and in two launches, in us, without scales and with: 2 tokens of
// 4096 x 4096 5.1, 6.7 and 5.7, 6.9; 4 of it 5.6, 6.9 and 6.4, 7.1; 8 of it 7.1, 7.1 and 8.6, 7.3; 4 of 6144 x 4096
// 7.4, 8.3 and 8.7, 8.5; 2 of 4096 x 11008 10.0, 9.6 and 11.7, 9.9; 16 of 8192 x 1024 4.8, 5.2 and 6.1, 5.5.
// (One token: wherever the product streams, at most 17632 columns, 9.3 KiB of LDS.)
bool mxfp4_linear_fused(int64_t T, int64_t M, int64_t cols) {
  return (T == 1 || (T <= 16 && T * cols <= 16384)) && mxfp4_form(T, M, (cols + 31) / 32 * 16) == kMxFew;
}

hipError_t launch_mxfp4_linear_fused(const MxArgs& a, const void* x, int64_t ldx, const float* s,
                                     int cols, hipStream_t stream) {
  if (a.T <= 0 || a.M <= 0) return hipSuccess;
  const MxFewArgs f{a, (const uint16_t*)x, s, ldx, cols};
  return a.T == 1   ? launch_few<1, 1>(f, stream)
         : a.T == 2 ? launch_few<2, 1>(f, stream)
                    : launch_few<4, 1>(f, stream);
}

}  // namespace awq
