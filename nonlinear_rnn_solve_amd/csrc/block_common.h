// block_common.h -- what the kernels of libpararnn_block.so share beyond lm_common.h: sequences packed along time, SiLU, and
// column sums of partial results in a fixed order.
#ifndef PARARNN_BLOCK_COMMON_H
#define PARARNN_BLOCK_COMMON_H

#include "lm_common.h"
#include "pararnn_block.h"

namespace lm {

// the sequences of a row: offsets (null: one sequence), their number and the row's steps
struct Seqs {
  const int32_t* cu;
  int64_t n, T;
  // first step of sequence j and the step after its last, within [0, T] whatever the offsets hold
  DEV int64_t clamp(int64_t t) const { return t < 0 ? 0 : t > T ? T : t; }
  DEV int64_t begin(int64_t j) const { return j > 0 ? clamp(cu[j]) : 0; }
  DEV int64_t end(int64_t j) const { return j + 1 < n ? clamp(cu[j + 1]) : T; }
  // the sequence that step t belongs to: the number of offsets cu[1 .. n-1] at or below t
  DEV int64_t of(int64_t t) const {
    int64_t lo = 0, hi = n - 1;
    while (lo < hi) {
      const int64_t mid = lo + (hi - lo + 1) / 2;
      if (cu[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  }
};

DEV float silu(float p) { return p * sigmoid(p); }
// d silu / dp, from p and its sigmoid
DEV float silu_slope(float p, float s) { return s * fmaf(p, 1.0f - s, 1.0f); }

// ---------------- column sums: the sum over rows of in[row][col], put where `out` has it, in one or two launches ----------------
constexpr int64_t kSumRows = 256;     // rows that one workgroup adds up where there are more than twice as many
inline int64_t colsum_groups(int64_t rows) { return rows > 2 * kSumRows ? ceil_div(rows, kSumRows) : 1; }
// floats of scratch for the sums of `rows` rows of `cols`
inline int64_t colsum_floats(int64_t rows, int64_t cols) {
  const int64_t g = colsum_groups(rows);
  return g > 1 ? g * cols : 0;
}
struct ToScratch {
  float* p;
  int64_t cols;
  DEV void operator()(int64_t group, int64_t col, float v) const { p[group * cols + col] = v; }
};

// 64 columns a workgroup, its four waves take every fourth row; sums in 64 bits, added in a fixed order
template <typename Out>
static __global__ __launch_bounds__(256) void k_colsum(const float* in, int64_t rows, int64_t cols, int64_t per, const Out out) {
  __shared__ double part[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t cblocks = (cols + 63) / 64, g = blockIdx.x / cblocks, col = (blockIdx.x - g * cblocks) * 64 + lane;
  const int64_t r0 = g * per, r1 = r0 + per < rows ? r0 + per : rows;
  double a0 = 0, a1 = 0;
  if (col < cols) {
    const float* p = in + (r0 + wave) * cols + col;
    int64_t r = r0 + wave;
    for (; r + 12 < r1; r += 16, p += 16 * cols) {
      const float x0 = p[0], x1 = p[4 * cols], x2 = p[8 * cols], x3 = p[12 * cols];
      a0 += static_cast<double>(x0) + x1;
      a1 += static_cast<double>(x2) + x3;
    }
    for (; r < r1; r += 4, p += 4 * cols) a0 += *p;
  }
  part[wave][lane] = a0 + a1;
  __syncthreads();
  if (wave == 0 && col < cols) out(g, col, static_cast<float>((part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane])));
}

// `scratch`: colsum_floats() floats.  rows = 0 gives zeros.  False: the launch would be too large.
template <typename Out>
inline bool colsum(const float* in, int64_t rows, int64_t cols, const Out& out, float* scratch, hipStream_t stream) {
  if (cols == 0) return true;
  const int64_t g = colsum_groups(rows), cb = ceil_div(cols, 64);
  if (!grid_ok(cb * g, 256)) return false;
  if (g > 1) {
    k_colsum<<<dim3(static_cast<uint32_t>(cb * g)), dim3(256), 0, stream>>>(in, rows, cols, kSumRows, ToScratch{scratch, cols});
    in = scratch;
    rows = g;
  }
  k_colsum<<<dim3(static_cast<uint32_t>(cb)), dim3(256), 0, stream>>>(in, rows, cols, rows, out);
  return true;
}

// a workspace of `need` bytes is there
inline bool ws_ok(const void* ws, size_t have, size_t need) { return need == 0 || (ws && aligned(ws, 256) && have >= need); }

}  // namespace lm
#endif
