// block_ffn.hip -- the gated feed-forward product of pararnn_block.h and its gradients.
//
//   g = x Wg^T, u = x Wu^T, h = act(g) u;   dg = dh u act'(g), du = dh act(g);
//   d_x = dg Wg + du Wu,  d_Wg = dg^T x,  d_Wu = du^T x

#include <algorithm>

#include "block_common.h"

namespace lm {

// ------------------------------------------------------------------------------------------------
// One matrix product serves all of them: C[m][n] = sum_k A[m][k] B[n][k], both operands dense along k.  The forward pass has
// them so as they are; for the gradients the pass that forms dg and du writes them transposed too, and x and the weights are
// transposed into the workspace, with k padded by zeros.
// ------------------------------------------------------------------------------------------------
using v16f = float __attribute__((ext_vector_type(16)));
using v4f = float __attribute__((ext_vector_type(4)));
using v8b = __bf16 __attribute__((ext_vector_type(8)));
using v4u = uint32_t __attribute__((ext_vector_type(4)));

constexpr int kKBytes = 128;    // of k in a tile: 64 bfloat16 or 32 float32
constexpr int kPad = 64;        // k of a transposed operand is a multiple of it

// activations and their slopes
template <int ACT> DEV float act(float g) {
  if constexpr (ACT == PARARNN_BLOCK_SILU) return g * sigmoid(g);
  // g Phi(g) ~ g sig(2 sqrt(2 / pi) (g + 0.044715 g^3))
  return g * sigmoid(1.5957691216057308f * fmaf(0.044715f * g, g * g, g));
}
template <int ACT> DEV float slope(float g) {
  if constexpr (ACT == PARARNN_BLOCK_SILU) {
    const float s = sigmoid(g);
    return silu_slope(g, s);
  }
  const float s = sigmoid(1.5957691216057308f * fmaf(0.044715f * g, g * g, g));
  return s * fmaf(g * (1.0f - s), 1.5957691216057308f * fmaf(3 * 0.044715f * g, g, 1.0f), 1.0f);
}

struct GemmArgs {
  const void *a, *b0, *b1;      // b1: the second weight (forward)
  int64_t sa, sb0, sb1;
  int64_t M, N, K;              // N: of one weight
  void *c0, *c1;                // rows from `split` on go to c1
  int64_t sc0, sc1, split;
  void* pre;
};

// 16 bytes of a row from element k on, zeros past its n elements or where the row is none
template <typename T> DEV v4u load16(const T* row, int64_t k, int64_t n, bool there) {
  constexpr int V = 16 / sizeof(T);
  const Vec<T, V> v = load_row<T, V>(row + k, there ? n - k : 0, T{});
  return v4u{v.w[0], v.w[1], v.w[2], v.w[3]};
}

// the products of 16 bytes of k of each lane: 32 rows by 32 columns, two lanes a row (their halves of k)
template <typename T> DEV void mma(const v4u& a, const v4u& b, v16f& c) {
  if constexpr (sizeof(T) == 2) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0, 0);
  } else {
    const v4f x = __builtin_bit_cast(v4f, a), y = __builtin_bit_cast(v4f, b);
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[j], y[j], c, 0, 0, 0);
  }
}
// row of value i of a lane's 16 (its column is the lane modulo 32)
DEV int row_of_acc(int i, int lane) { return 8 * (i / 4) + 4 * (lane / 32) + i % 4; }

// A workgroup of four waves forms 128 by 128 of C (forward: 128 by 64 of both products), each wave 64 by 64.  The next
// tile's rows are in registers while this one is multiplied from shared memory; its 16-byte pieces are exchanged within a row by the row's
// number, so that no two of the eight lanes that read together meet in a bank.  Any alignment and size.
template <typename T, bool GATED, int ACT>
__global__ __launch_bounds__(256) void k_gemm(const GemmArgs p, uint32_t mtiles) {
  constexpr int V = 16 / sizeof(T), BK = kKBytes / sizeof(T);
  __shared__ v4u sa[128][8], sb[128][8];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave & 1, wn = wave >> 1;
  const int64_t mt = blockIdx.x % mtiles, nt = blockIdx.x / mtiles;
  const int64_t m0 = mt * 128, n0 = nt * (GATED ? 64 : 128);
  const T* a = static_cast<const T*>(p.a);
  v4u ra[4], rb[4];
  const auto load = [&](int64_t k0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int id = threadIdx.x + i * 256, r = id / 8, c = id % 8;
      ra[i] = load16<T>(a + (m0 + r) * p.sa, k0 + c * V, p.K, m0 + r < p.M);
      const bool second = GATED && r >= 64;
      const int64_t n = n0 + (second ? r - 64 : r);
      const T* b = static_cast<const T*>(second ? p.b1 : p.b0);
      rb[i] = load16<T>(b + n * (second ? p.sb1 : p.sb0), k0 + c * V, p.K, n < p.N);
    }
  };
  v16f acc[2][2] = {};
  load(0);
  for (int64_t k0 = 0; k0 < p.K; k0 += BK) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int id = threadIdx.x + i * 256, r = id / 8, c = id % 8;
      sa[r][c ^ (r & 7)] = ra[i];
      sb[r][c ^ (r & 7)] = rb[i];
    }
    __syncthreads();
    if (k0 + BK < p.K) load(k0 + BK);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      v4u fa[2], fb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = wm * 64 + i * 32 + (lane & 31);
        // gated: 32 columns of the gate, then the same of the other product
        const int n = GATED ? i * 64 + wn * 32 + (lane & 31) : wn * 64 + i * 32 + (lane & 31);
        const int c = kk * 2 + lane / 32;
        fa[i] = sa[r][c ^ (r & 7)];
        fb[i] = sb[n][c ^ (n & 7)];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) mma<T>(fa[i], fb[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int64_t m = m0 + wm * 64 + i * 32 + row_of_acc(e, lane);
      if (m >= p.M) continue;
      if constexpr (GATED) {
        const int64_t n = n0 + wn * 32 + (lane & 31);
        if (n >= p.N) continue;
        const float g = acc[i][0][e], u = acc[i][1][e];
        static_cast<T*>(p.c0)[m * p.sc0 + n] = from_f32<T>(act<ACT>(g) * u);
        if (p.pre) {
          T* pre = static_cast<T*>(p.pre) + m * 2 * p.N + n;
          pre[0] = from_f32<T>(g);
          pre[p.N] = from_f32<T>(u);
        }
      } else {
        T* c = m < p.split ? static_cast<T*>(p.c0) + m * p.sc0 : static_cast<T*>(p.c1) + (m - p.split) * p.sc1;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int64_t n = n0 + wn * 64 + j * 32 + (lane & 31);
          if (n < p.N) c[n] = from_f32<T>(acc[i][j][e]);
        }
      }
    }
}

// ---------------- what the gradients' products are made of ----------------
// dg and du of R rows as [R][2 F] and as [2 F][Rp], zeros from R to Rp; 64 by 64 of each a workgroup
struct SplitArgs {
  const void *pre, *dh;
  int64_t sdh, R, F, Rp, Fp2;   // Fp2: row stride of `rows`
  void *rows, *cols;
};
template <typename T, int ACT> __global__ __launch_bounds__(256) void k_ffn_split(const SplitArgs p, uint32_t rtiles) {
  __shared__ T tg[64][65], tu[64][65];
  const int64_t r0 = static_cast<int64_t>(blockIdx.x % rtiles) * 64, f0 = static_cast<int64_t>(blockIdx.x / rtiles) * 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const int64_t r = r0 + wave * 16 + i, f = f0 + lane;
    float dg = 0.0f, du = 0.0f;
    if (r < p.R && f < p.F) {
      const T* pre = static_cast<const T*>(p.pre) + r * 2 * p.F + f;
      const float g = to_f32(pre[0]), u = to_f32(pre[p.F]), dh = to_f32(static_cast<const T*>(p.dh)[r * p.sdh + f]);
      dg = dh * u * slope<ACT>(g);
      du = dh * act<ACT>(g);
      if (p.rows) {
        T* to = static_cast<T*>(p.rows) + r * p.Fp2 + f;
        to[0] = from_f32<T>(dg);
        to[p.F] = from_f32<T>(du);
      }
    }
    tg[wave * 16 + i][lane] = from_f32<T>(dg);
    tu[wave * 16 + i][lane] = from_f32<T>(du);
  }
  if (!p.cols) return;
  __syncthreads();
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const int64_t f = f0 + wave * 16 + i, r = r0 + lane;
    if (f < p.F && r < p.Rp) {
      T* to = static_cast<T*>(p.cols) + f * p.Rp + r;
      to[0] = tg[lane][wave * 16 + i];
      to[p.F * p.Rp] = tu[lane][wave * 16 + i];
    }
  }
}

// to[c][r] = from[r][c] for R rows of C, zeros for r from R to Rp; `to` has row stride st
template <typename T>
__global__ __launch_bounds__(256) void k_transpose(const T* from, int64_t sf, int64_t R, int64_t C, T* to, int64_t st, int64_t Rp,
                                                   uint32_t rtiles) {
  __shared__ T tile[64][65];
  const int64_t r0 = static_cast<int64_t>(blockIdx.x % rtiles) * 64, c0 = static_cast<int64_t>(blockIdx.x / rtiles) * 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const int64_t r = r0 + wave * 16 + i, c = c0 + lane;
    tile[wave * 16 + i][lane] = r < R && c < C ? from[r * sf + c] : T{};
  }
  __syncthreads();
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const int64_t c = c0 + wave * 16 + i, r = r0 + lane;
    if (c < C && r < Rp) to[c * st + r] = tile[lane][wave * 16 + i];
  }
}

// ---------------- host ----------------
inline int64_t padded(int64_t n) { return ceil_div(n, kPad) * kPad; }
template <typename T, bool GATED, int ACT> static bool gemm(const GemmArgs& p, hipStream_t st) {
  const int64_t mt = ceil_div(p.M, 128), nt = ceil_div(p.N, GATED ? 64 : 128);
  if (mt == 0 || nt == 0) return true;
  if (!grid_ok(mt * nt, 256)) return false;
  k_gemm<T, GATED, ACT><<<dim3(static_cast<uint32_t>(mt * nt)), dim3(256), 0, st>>>(p, static_cast<uint32_t>(mt));
  return true;
}
template <typename T> static bool transpose(const void* from, int64_t sf, int64_t R, int64_t C, T* to, int64_t st, int64_t Rp,
                                            hipStream_t stream) {
  const int64_t rt = ceil_div(Rp, 64), ct = ceil_div(C, 64);
  if (rt == 0 || ct == 0) return true;
  if (!grid_ok(rt * ct, 256)) return false;
  k_transpose<T><<<dim3(static_cast<uint32_t>(rt * ct)), dim3(256), 0, stream>>>(static_cast<const T*>(from), sf, R, C, to, st, Rp,
                                                                                 static_cast<uint32_t>(rt));
  return true;
}

constexpr int64_t kMost = INT32_MAX - 512;
static bool sizes_ok(int64_t R, int64_t D, int64_t F) {
  return R >= 0 && D >= 0 && F >= 0 && (R > kMost || D > kMost || F > kMost || (sizes_fit(R, D) && sizes_fit(R, F, 2) && sizes_fit(F, D, 2)));
}
// elements of the gradient's workspace: d_pre [R][F2], d_pre^T [2 F][Rp], x^T [D][Rp], weights^T [D][F2]
struct GradRoom {
  int64_t F2, Rp, rows, cols, xt, wt;
  int64_t total() const { return rows + cols + xt + wt; }
};
static GradRoom grad_room(int64_t R, int64_t D, int64_t F) {
  GradRoom g;
  g.F2 = padded(2 * F), g.Rp = padded(R);
  g.rows = padded(R * g.F2), g.cols = padded(2 * F * g.Rp), g.xt = padded(D * g.Rp), g.wt = padded(D * g.F2);
  return g;
}

template <typename T, int ACT>
static pararnn_status backward(int64_t R, int64_t D, int64_t F, const void* x, int64_t sx, const void* wg, int64_t sg, const void* wu,
                               int64_t su, const void* pre, const void* dh, int64_t sdh, void* dx, int64_t sdx, void* dwg,
                               int64_t sdg, void* dwu, int64_t sdu, T* ws, hipStream_t st) {
  const GradRoom room = grad_room(R, D, F);
  T *rows = ws, *cols = rows + room.rows, *xt = cols + room.cols, *wt = xt + room.xt;
  const int64_t rt = ceil_div(room.Rp, 64), ft = ceil_div(F, 64);
  if (!grid_ok(rt * ft, 256)) return PARARNN_ERR_UNSUPPORTED;
  bool ok = true;
  if (rt * ft) {
    const SplitArgs s{pre, dh, sdh, R, F, room.Rp, room.F2, dx ? rows : nullptr, dwg ? cols : nullptr};
    k_ffn_split<T, ACT><<<dim3(static_cast<uint32_t>(rt * ft)), dim3(256), 0, st>>>(s, static_cast<uint32_t>(rt));
  }
  if (dx && R && D) {
    // the columns between 2 F and its padding are read by no product: k ends at 2 F
    ok = ok && transpose<T>(wg, sg, F, D, wt, room.F2, F, st) && transpose<T>(wu, su, F, D, wt + F, room.F2, F, st);
    GemmArgs p{rows, wt, nullptr, room.F2, room.F2, 0, R, D, 2 * F, dx, nullptr, sdx, 0, R, nullptr};
    ok = ok && gemm<T, false, 0>(p, st);
  }
  if (dwg && F && D) {
    ok = ok && transpose<T>(x, sx, R, D, xt, room.Rp, room.Rp, st);
    GemmArgs p{cols, xt, nullptr, room.Rp, room.Rp, 0, 2 * F, D, R, dwg, dwu, sdg, sdu, F, nullptr};
    ok = ok && gemm<T, false, 0>(p, st);
  }
  return ok ? launched() : PARARNN_ERR_UNSUPPORTED;
}

}  // namespace lm

using namespace lm;

extern "C" size_t pararnn_block_gated_linear_workspace_bytes(int dtype, int64_t R, int64_t D, int64_t F, int gradient) {
  if (!dtype_ok(dtype) || !sizes_ok(R, D, F) || R > kMost || D > kMost || F > kMost) return 0;
  return gradient ? static_cast<size_t>(grad_room(R, D, F).total()) * dtype_size(dtype) : 0;
}

extern "C" pararnn_status pararnn_block_gated_linear(int dtype, int act, int64_t R, int64_t D, int64_t F, const void* x,
                                                     int64_t x_stride, const void* w_gate, int64_t gate_stride, const void* w_up,
                                                     int64_t up_stride, void* h, int64_t h_stride, void* pre, void* ws,
                                                     size_t ws_bytes, void* stream) {
  if (!dtype_ok(dtype) || (act != PARARNN_BLOCK_SILU && act != PARARNN_BLOCK_GELU) || !sizes_ok(R, D, F))
    return PARARNN_ERR_INVALID_ARG;
  const size_t e = dtype_size(dtype);
  if (!ptr_ok(x, e, R > 0 && D > 0) || !ptr_ok(w_gate, e, F > 0 && D > 0) || !ptr_ok(w_up, e, F > 0 && D > 0) ||
      !ptr_ok(h, e, R > 0 && F > 0) || !ptr_ok(pre, e, false) || !plane_ok(R, x_stride) || !plane_ok(F, gate_stride) ||
      !plane_ok(F, up_stride) || !plane_ok(R, h_stride))
    return PARARNN_ERR_INVALID_ARG;
  if (R > kMost || D > kMost || F > kMost) return PARARNN_ERR_UNSUPPORTED;
  if (!ws_ok(ws, ws_bytes, pararnn_block_gated_linear_workspace_bytes(dtype, R, D, F, 0))) return PARARNN_ERR_WORKSPACE;
  if (R == 0 || F == 0) return PARARNN_OK;
  const GemmArgs p{x, w_gate, w_up, x_stride, gate_stride, up_stride, R, F, D, h, nullptr, h_stride, 0, R, pre};
  const auto st = static_cast<hipStream_t>(stream);
  bool ok;
  if (dtype == PARARNN_BF16)
    ok = act == PARARNN_BLOCK_SILU ? gemm<bf16, true, PARARNN_BLOCK_SILU>(p, st) : gemm<bf16, true, PARARNN_BLOCK_GELU>(p, st);
  else
    ok = act == PARARNN_BLOCK_SILU ? gemm<float, true, PARARNN_BLOCK_SILU>(p, st) : gemm<float, true, PARARNN_BLOCK_GELU>(p, st);
  return ok ? launched() : PARARNN_ERR_UNSUPPORTED;
}

extern "C" pararnn_status pararnn_block_gated_linear_vjp(int dtype, int act, int64_t R, int64_t D, int64_t F, const void* x,
                                                         int64_t x_stride, const void* w_gate, int64_t gate_stride, const void* w_up,
                                                         int64_t up_stride, const void* pre, const void* dh, int64_t dh_stride,
                                                         void* d_x, int64_t d_x_stride, void* d_w_gate, int64_t d_gate_stride,
                                                         void* d_w_up, int64_t d_up_stride, void* ws, size_t ws_bytes, void* stream) {
  if (!dtype_ok(dtype) || (act != PARARNN_BLOCK_SILU && act != PARARNN_BLOCK_GELU) || !sizes_ok(R, D, F))
    return PARARNN_ERR_INVALID_ARG;
  const size_t e = dtype_size(dtype);
  if (!ptr_ok(x, e, R > 0 && D > 0) || !ptr_ok(w_gate, e, F > 0 && D > 0) || !ptr_ok(w_up, e, F > 0 && D > 0) ||
      !ptr_ok(pre, e, R > 0 && F > 0) || !ptr_ok(dh, e, R > 0 && F > 0) || !ptr_ok(d_x, e, false) || !ptr_ok(d_w_gate, e, false) ||
      !ptr_ok(d_w_up, e, false) || (d_w_gate == nullptr) != (d_w_up == nullptr) || !plane_ok(R, x_stride) ||
      !plane_ok(F, gate_stride) || !plane_ok(F, up_stride) || !plane_ok(R, dh_stride) || !plane_ok(R, d_x_stride) ||
      !plane_ok(F, d_gate_stride) || !plane_ok(F, d_up_stride))
    return PARARNN_ERR_INVALID_ARG;
  if (R > kMost || D > kMost || F > kMost) return PARARNN_ERR_UNSUPPORTED;
  if (!ws_ok(ws, ws_bytes, pararnn_block_gated_linear_workspace_bytes(dtype, R, D, F, 1))) return PARARNN_ERR_WORKSPACE;
  if (!d_x && !d_w_gate) return PARARNN_OK;
  const auto st = static_cast<hipStream_t>(stream);
  const auto run = [&](auto t, auto a) {
    using T = decltype(t);
    return backward<T, decltype(a)::value>(R, D, F, x, x_stride, w_gate, gate_stride, w_up, up_stride, pre, dh, dh_stride, d_x,
                                           d_x_stride, d_w_gate, d_gate_stride, d_w_up, d_up_stride, static_cast<T*>(ws), st);
  };
  using Silu = std::integral_constant<int, PARARNN_BLOCK_SILU>;
  using Gelu = std::integral_constant<int, PARARNN_BLOCK_GELU>;
  if (dtype == PARARNN_BF16) return act == PARARNN_BLOCK_SILU ? run(bf16{}, Silu{}) : run(bf16{}, Gelu{});
  return act == PARARNN_BLOCK_SILU ? run(0.0f, Silu{}) : run(0.0f, Gelu{});
}
