// Rows of 8-bit integers: step[r] = max_i |v[r][i]| / 127, code[r][i] = rint(v[r][i] / step[r])
// with v = A, A / s or A * s.
//
// Pages: "AWQ" scholia-log notes §2.3 (symmetric quantiser: scale to the largest magnitude,
// round) and §4.3 (S^-1 folded into the activations).
//
// One block a row, bound by reading A from HBM: a thread keeps its values in registers
// between the maximum and the rounding, so A is read once (rows too long for that are read
// a second time, from cache).  4096 rows of 4096 divided by a scale a column: 19.5 us, 2.6 TB/s
// (a copy of as many bytes takes 10): each value takes two correctly rounded operations, the
// fold's division and a quotient by the step.
#include <hip/hip_runtime.h>

#include "grid.h"
#include "int8_quant.h"
#include "serve_internal.h"

namespace awq {

namespace {

constexpr int kRowThreads = 256;

// NCH: 8-column chunks a thread keeps in registers (0: reads the row twice).
template <bool BF16, bool VEC, int NCH>
__global__ __launch_bounds__(kRowThreads) void k_int8_rows(
    const uint16_t* __restrict__ A, unsigned rows, int K, int64_t lda, const float* __restrict__ s, int fold,
    int8_t* __restrict__ codes, int64_t ldc, float* __restrict__ steps) {
  __shared__ uint32_t red[kRowThreads / 64];
  const unsigned number = block_number();
  if (number >= rows) return;  // the whole block
  const int64_t row = number;
  const int tid = threadIdx.x;
  const uint16_t* a = A + row * lda;
  const int nch = ((K + 15) / 16) * 2;  // 8-column chunks, whole 16-byte groups of codes
  float v[NCH > 0 ? NCH : 1][8];
  uint32_t top = 0;
  if constexpr (NCH > 0) {
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int ch = tid + c * kRowThreads;
      if (ch < nch) {
        load_row8<BF16, VEC>(a, s, fold, 8 * ch, K, v[c]);
        top = max_abs8(v[c], top);
      }
    }
  } else {
    for (int ch = tid; ch < nch; ch += kRowThreads) {
      load_row8<BF16, VEC>(a, s, fold, 8 * ch, K, v[0]);
      top = max_abs8(v[0], top);
    }
  }
  top = block_max<kRowThreads / 64>(top, red);
  const RowStep st = row_step(top);
  if (tid == 0) steps[row] = st.step;
  int8_t* out = codes + row * ldc;
  if constexpr (NCH > 0) {
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int ch = tid + c * kRowThreads;
      if (ch < nch) *(uint2*)(out + 8 * ch) = row_codes8(v[c], st);
    }
  } else {
    for (int ch = tid; ch < nch; ch += kRowThreads) {
      load_row8<BF16, VEC>(a, s, fold, 8 * ch, K, v[0]);
      *(uint2*)(out + 8 * ch) = row_codes8(v[0], st);
    }
  }
}

}  // namespace

hipError_t launch_int8_rows(const void* A, int64_t rows, int cols, int64_t lda, bool bf16,
                            const float* s, int fold, int8_t* codes, int64_t ld_codes,
                            float* steps, hipStream_t stream) {
  if (rows <= 0) return hipSuccess;
  const bool vec = row_vector_loads(A, lda, s);
  const int nch = ((cols + 15) / 16) * 2;
  // registers hold 2 or 8 chunks of 8 columns a thread: rows of up to 4096 or 16384 columns
  const int keep = nch <= 2 * kRowThreads ? 2 : nch <= 8 * kRowThreads ? 8 : 0;
  const int f = s ? fold : kFoldNone;
#define AWQ_ROWS(B, V, N)                                                                     \
  hipLaunchKernelGGL((k_int8_rows<B, V, N>), grid_of(rows), dim3(kRowThreads), 0, stream, \
                     (const uint16_t*)A, (unsigned)rows, cols, lda, s, f, codes, ld_codes, steps)
#define AWQ_ROWS_N(B, V)            \
  switch (keep) {                   \
    case 2: AWQ_ROWS(B, V, 2); break; \
    case 8: AWQ_ROWS(B, V, 8); break; \
    default: AWQ_ROWS(B, V, 0); break; \
  }
  if (bf16) {
    if (vec) { AWQ_ROWS_N(true, true) } else { AWQ_ROWS_N(true, false) }
  } else {
    if (vec) { AWQ_ROWS_N(false, true) } else { AWQ_ROWS_N(false, false) }
  }
#undef AWQ_ROWS_N
#undef AWQ_ROWS
  return hipGetLastError();
}

}  // namespace awq
