// lm_norm.hip -- layer normalisation of pararnn_lm.h and its gradients.
//
// Both directions are bound by memory: a row is read once into registers (up to 16 columns a lane), reduced there and
// written.  The mean comes first and the variance is summed about it, since the row is at hand.  Measured, bf16 8192 x 4096
// with residual: forward 51.6 us (268 MB, 5.2 TB/s), gradient 53.6 us (268 MB and 17 MB of parts, 5.3 TB/s) and 4.7 us for the
// parameter sums; float32 5001 x 2047 15, 22.7 and 4.2 us.  A copy runs at 5.1 TB/s.

#include <algorithm>
#include <type_traits>

#include "lm_common.h"

namespace lm {

// A row is held by LPR lanes (16, 64, 256 or 1024) of CPL columns each (8 or 16), in vectors of 16 bytes: vector k of lane l
// is columns (k LPR + l) V and on.
template <typename T, int LPR_, int CPL_> struct Shape {
  static constexpr int LPR = LPR_, CPL = CPL_, V = 16 / sizeof(T), NV = CPL / V;
};

// Sums of K values over the LPR lanes of a row, the same for each of them: lanes, then (LPR > 64) waves in order through
// shared memory, which alternates between two sets so that one barrier a call is enough.  Every thread of the workgroup
// calls it.
template <int LPR, int K, int NT> struct RowSum {
  static constexpr int WPR = LPR > WAVE ? LPR / WAVE : 1;
  float sh[LPR > WAVE ? 2 : 1][K][LPR > WAVE ? NT / WAVE : 1];
};
template <int LPR, int K, int NT> DEV void row_sums(float (&v)[K], RowSum<LPR, K, NT>& s, int& turn) {
  if constexpr (LPR == 16) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = row_sum(v[k]);
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = wave_sum(v[k]);
    if constexpr (LPR > WAVE) {
      const int wave = threadIdx.x / WAVE, first = wave / s.WPR * s.WPR;
      if (threadIdx.x % WAVE == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) s.sh[turn][k][wave] = v[k];
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k) {
        v[k] = s.sh[turn][k][first];
#pragma unroll
        for (int w = 1; w < s.WPR; ++w) v[k] += s.sh[turn][k][first + w];
      }
      turn ^= 1;
    }
  }
}

struct NormArgs {
  const void *x, *res;
  const float *weight, *bias;
  void *y, *sum;
  float* stats;
  int64_t sx, sres, sy, ssum, N, D;
  float eps;
};

template <typename T, class S, int NT>
__global__ __launch_bounds__(NT) void k_norm(const NormArgs p) {
  constexpr int LPR = S::LPR, V = S::V, NV = S::NV;
  __shared__ RowSum<LPR, 1, NT> sh;
  int turn = 0;
  const int lane = threadIdx.x % LPR;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * (NT / LPR) + threadIdx.x / LPR;
  const bool on = n < p.N;
  const T* x = static_cast<const T*>(p.x) + (on ? n : 0) * p.sx;
  const T* res = p.res ? static_cast<const T*>(p.res) + (on ? n : 0) * p.sres : nullptr;
  float v[NV][V];
  {
    Vec<T, V> a[NV], b[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int64_t c = static_cast<int64_t>(k * LPR + lane) * V;
      a[k] = load_row<T, V>(x + c, p.D - c, T{});
      if (res) b[k] = load_row<T, V>(res + c, p.D - c, T{});
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int64_t c = static_cast<int64_t>(k * LPR + lane) * V;
#pragma unroll
      for (int e = 0; e < V; ++e) v[k][e] = a[k].get(e);
      if (res) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[k][e] = to_f32(from_f32<T>(v[k][e] + b[k].get(e)));
        if (on) store_row<T, V>(static_cast<T*>(p.sum) + n * p.ssum + c, p.D - c, v[k]);
      }
    }
  }
  float s[1] = {0.0f};
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) s[0] += v[k][e];   // columns past D are 0
  row_sums(s, sh, turn);
  const float mean = s[0] / static_cast<float>(p.D);
  s[0] = 0.0f;
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      v[k][e] = (k * LPR + lane) * V + e < p.D ? v[k][e] - mean : 0.0f;
      s[0] = fmaf(v[k][e], v[k][e], s[0]);
    }
  row_sums(s, sh, turn);
  if (!on) return;
  const float rstd = 1.0f / sqrtf(s[0] / static_cast<float>(p.D) + p.eps);
  T* y = static_cast<T*>(p.y) + n * p.sy;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int64_t c = static_cast<int64_t>(k * LPR + lane) * V;
    if (c >= p.D) break;
    float o[V];
    const Vec<float, V> w = load_row<float, V>(p.weight + c, p.D - c, 0.0f);
    Vec<float, V> b{};
    if (p.bias) b = load_row<float, V>(p.bias + c, p.D - c, 0.0f);
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = fmaf(v[k][e] * rstd, w.get(e), b.get(e));
    store_row<T, V>(y + c, p.D - c, o);
  }
  if (p.stats && lane == 0) {
    p.stats[2 * n] = mean;
    p.stats[2 * n + 1] = rstd;
  }
}

struct NormGradArgs {
  const void *dy, *s, *dsum;
  const float *weight, *stats;
  void* dx;
  int64_t sdy, ss, sdsum, sdx, N, D;
  float* part;   // [workgroups][2][D] sums of dy n and of dy over a workgroup's rows, or null
};

// A workgroup takes NT / LPR rows at a time, as many workgroups as the chip holds at once in turn, and keeps the parameter sums of its lanes'
// columns in registers; in the end its row groups' are added up in order, those of a wave by lane exchanges, then the
// PG waves (or groups of waves) of different rows through shared memory, kStage columns a lane at a time.
// 512 threads and 512 workgroups against 1024 and 256: bf16 8192 x 4096 53.6 and 54.6 us, 20000 x 700 33.8 and 34.4, 3 x 552
// 4.3 and 5.2; 256 threads 55.6 and 35.0, and twice the time for their sums.  What a lane keeps over a row's reduction are
// the normalised values and dy weight, in the registers of what was loaded: nothing spills (60 us where it did).
constexpr int kGradAll = 1 << 18, kStage = 4;
constexpr int grad_threads(int64_t lpr) { return lpr > 512 ? 1024 : 512; }
template <typename T, class S>
__global__ __launch_bounds__(grad_threads(S::LPR)) void k_norm_grad(const NormGradArgs p) {
  constexpr int LPR = S::LPR, V = S::V, NV = S::NV, NT = grad_threads(S::LPR), RG = NT / LPR;
  constexpr int PL = LPR < WAVE ? WAVE : LPR, PG = NT / PL;
  __shared__ RowSum<LPR, 2, NT> sh;
  __shared__ float sh_p[PG > 1 ? PG : 1][2][PG > 1 ? LPR * kStage : 1];
  int turn = 0;
  const int lane = threadIdx.x % LPR, group = threadIdx.x / LPR;
  const float inv = 1.0f / static_cast<float>(p.D);
  float sw[NV][V], sb[NV][V];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) sw[k][e] = sb[k][e] = 0.0f;
  for (int64_t n0 = static_cast<int64_t>(blockIdx.x) * RG; n0 < p.N; n0 += static_cast<int64_t>(gridDim.x) * RG) {
    const int64_t n = n0 + group < p.N ? n0 + group : p.N - 1;
    const bool on = n0 + group < p.N;
    const T* dy = static_cast<const T*>(p.dy) + n * p.sdy;
    const T* s = static_cast<const T*>(p.s) + n * p.ss;
    const T* dsum = p.dsum ? static_cast<const T*>(p.dsum) + n * p.sdsum : nullptr;
    Vec<T, V> a[NV], g[NV], ds[NV];
    Vec<float, V> w[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int64_t c = static_cast<int64_t>(k * LPR + lane) * V;
      a[k] = load_row<T, V>(s + c, p.D - c, T{});
      g[k] = load_row<T, V>(dy + c, p.D - c, T{});
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int64_t c = static_cast<int64_t>(k * LPR + lane) * V;
      if (dsum) ds[k] = load_row<T, V>(dsum + c, p.D - c, T{});
      w[k] = load_row<float, V>(p.weight + c, p.D - c, 0.0f);
    }
    const float mean = p.stats[2 * n], rstd = p.stats[2 * n + 1];
    float c12[2] = {0.0f, 0.0f};
    float xn[NV][V], t[NV][V];   // in the registers of s, dy and the weights
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = g[k].get(e);   // past D: 0
        xn[k][e] = (a[k].get(e) - mean) * rstd;
        t[k][e] = d * w[k].get(e);
        c12[0] += t[k][e];
        c12[1] = fmaf(t[k][e], xn[k][e], c12[1]);
        if (on) {
          sw[k][e] = fmaf(d, xn[k][e], sw[k][e]);
          sb[k][e] += d;
        }
      }
    row_sums(c12, sh, turn);
    const float c1 = c12[0] * inv, c2 = c12[1] * inv;
    if (on) {
      T* dx = static_cast<T*>(p.dx) + n * p.sdx;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int64_t c = static_cast<int64_t>(k * LPR + lane) * V;
        float o[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          o[e] = rstd * ((t[k][e] - c1) - xn[k][e] * c2);
          if (dsum) o[e] += ds[k].get(e);
        }
        store_row<T, V>(dx + c, p.D - c, o);
      }
    }
  }
  if (!p.part) return;
  if constexpr (PG > 1) {
    const int place = threadIdx.x / PL;
    float* out = p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.D;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int e0 = 0; e0 < V; e0 += kStage) {
#pragma unroll
        for (int e = 0; e < kStage; ++e) {
          float w = sw[k][e0 + e], b = sb[k][e0 + e];
#pragma unroll
          for (int o = LPR; o < WAVE; o <<= 1) {
            w += __shfl_xor(w, o, WAVE);
            b += __shfl_xor(b, o, WAVE);
          }
          if (threadIdx.x % PL < LPR) {
            sh_p[place][0][lane * kStage + e] = w;
            sh_p[place][1][lane * kStage + e] = b;
          }
        }
        __syncthreads();
        for (int at = threadIdx.x; at < 2 * LPR * kStage; at += NT) {
          const int which = at / (LPR * kStage), c = at % (LPR * kStage);
          float t = sh_p[0][which][c];
#pragma unroll
          for (int g = 1; g < PG; ++g) t += sh_p[g][which][c];
          const int64_t col = static_cast<int64_t>(k * LPR + c / kStage) * V + e0 + c % kStage;
          if (col < p.D) out[which * p.D + col] = t;
        }
        __syncthreads();
      }
  } else {
    float* out = p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.D;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int64_t c = static_cast<int64_t>(k * LPR + lane) * V;
      store_row<float, V>(out + c, p.D - c, sw[k]);
      store_row<float, V>(out + p.D + c, p.D - c, sb[k]);
    }
  }
}

// the workgroups' parts [rows][2][D] as d_weight and d_bias: a wave sums every 16th row, eight loads at a time, the
// waves' sums are added in order
__global__ __launch_bounds__(1024) void k_norm_params(const float* part, int64_t rows, int64_t D, float* dweight, float* dbias) {
  __shared__ float sh[16][WAVE];
  const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * WAVE + lane, cc = c < 2 * D ? c : 0;
  float s = 0.0f;
  for (int64_t n = wave; n < rows; n += 16 * 8) {
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = n + u * 16 < rows ? part[(n + u * 16) * 2 * D + cc] : 0.0f;
#pragma unroll
    for (int u = 0; u < 8; ++u) s += v[u];
  }
  sh[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || c >= 2 * D) return;
  s = 0.0f;
#pragma unroll
  for (int w = 0; w < 16; ++w) s += sh[w][lane];
  float* out = c < D ? dweight : dbias;
  if (out) out[c < D ? c : c - D] = s;
}

// calls f with the shape that holds D columns
template <typename T, class F> static void shape_of(int64_t D, F f) {
  const auto lanes = [&](auto lpr) {
    constexpr int L = decltype(lpr)::value;
    if (D <= L * 8) f(Shape<T, L, 8>{});
    else f(Shape<T, L, 16>{});
  };
  if (D <= 256) lanes(std::integral_constant<int, 16>{});
  else if (D <= 1024) lanes(std::integral_constant<int, 64>{});
  else if (D <= 4096) lanes(std::integral_constant<int, 256>{});
  else lanes(std::integral_constant<int, 1024>{});
}

// lanes of a row, threads of a workgroup of k_norm
static int64_t norm_threads(int64_t D) { return D <= 256 ? 16 : D <= 1024 ? 64 : D <= 4096 ? 256 : 1024; }
constexpr int norm_block(int64_t lanes) { return lanes > 256 ? 1024 : 256; }
// k_norm's launch holds N rows, the last workgroup's idle lanes included
static bool rows_ok(int64_t N, int64_t D) {
  const int64_t lanes = norm_threads(D), threads = norm_block(lanes);
  return grid_ok(ceil_div(N, threads / lanes), threads);
}
static int64_t grad_groups(int64_t N, int64_t D) {
  const int64_t lanes = norm_threads(D), threads = grad_threads(lanes);
  return std::min<int64_t>(ceil_div(N, threads / lanes), kGradAll / threads);
}

}  // namespace lm

using namespace lm;

extern "C" pararnn_status pararnn_lm_layer_norm(int dtype, int64_t N, int64_t D, const void* x, int64_t x_stride,
                                                const void* residual, int64_t residual_stride, const float* weight,
                                                const float* bias, float eps, void* y, int64_t y_stride, void* sum,
                                                int64_t sum_stride, float* stats, void* stream) {
  if (!dtype_ok(dtype) || !sizes_fit(N, D) || !(eps >= 0.0f)) return PARARNN_ERR_INVALID_ARG;
  if ((residual == nullptr) != (sum == nullptr)) return PARARNN_ERR_INVALID_ARG;
  if (N == 0 || D == 0) return PARARNN_OK;
  const size_t es = dtype_size(dtype);
  if (!ptr_ok(x, es) || !ptr_ok(residual, es, false) || !ptr_ok(weight, 4) || !ptr_ok(bias, 4, false) ||
      !ptr_ok(y, es) || !ptr_ok(sum, es, false) || !ptr_ok(stats, 4, false))
    return PARARNN_ERR_INVALID_ARG;
  if (!plane_ok(N, x_stride) || !plane_ok(N, y_stride) || (residual && (!plane_ok(N, residual_stride) || !plane_ok(N, sum_stride))))
    return PARARNN_ERR_INVALID_ARG;
  if (D > PARARNN_LM_NORM_MAX_D || !rows_ok(N, D)) return PARARNN_ERR_UNSUPPORTED;
  const NormArgs a{x, residual, weight, bias, y, sum, stats, x_stride, residual_stride, y_stride, sum_stride, N, D, eps};
  hipStream_t st = static_cast<hipStream_t>(stream);
  const auto run = [&](auto t) {
    using T = decltype(t);
    shape_of<T>(D, [&](auto s) {
      using S = decltype(s);
      constexpr int NT = norm_block(S::LPR);
      k_norm<T, S, NT><<<static_cast<unsigned>(ceil_div(N, NT / S::LPR)), NT, 0, st>>>(a);
    });
  };
  if (dtype == PARARNN_BF16) run(bf16{});
  else run(float{});
  return launched();
}

extern "C" size_t pararnn_lm_layer_norm_vjp_workspace_bytes(int64_t N, int64_t D) {
  if (!sizes_fit(N, D) || !sizes_fit(1024, D)) return 0;
  return static_cast<size_t>(grad_groups(N, D) * 2 * D * 4 + 256);
}

extern "C" pararnn_status pararnn_lm_layer_norm_vjp(int dtype, int64_t N, int64_t D, const void* dy, int64_t dy_stride,
                                                    const void* s, int64_t s_stride, const float* weight,
                                                    const float* stats, const void* d_sum, int64_t d_sum_stride,
                                                    void* d_x, int64_t d_x_stride, float* d_weight, float* d_bias,
                                                    void* ws, size_t ws_bytes, void* stream) {
  if (!dtype_ok(dtype) || !sizes_fit(N, D)) return PARARNN_ERR_INVALID_ARG;
  if (!ptr_ok(d_weight, 4, false) || !ptr_ok(d_bias, 4, false)) return PARARNN_ERR_INVALID_ARG;
  if (D == 0) return PARARNN_OK;
  const size_t es = dtype_size(dtype);
  if (N > 0 && (!ptr_ok(dy, es) || !ptr_ok(s, es) || !ptr_ok(weight, 4) || !ptr_ok(stats, 4) ||
                !ptr_ok(d_sum, es, false) || !ptr_ok(d_x, es)))
    return PARARNN_ERR_INVALID_ARG;
  if (!plane_ok(N, dy_stride) || !plane_ok(N, s_stride) || !plane_ok(N, d_x_stride) || (d_sum && !plane_ok(N, d_sum_stride)))
    return PARARNN_ERR_INVALID_ARG;
  if (D > PARARNN_LM_NORM_MAX_D || !rows_ok(N, D)) return PARARNN_ERR_UNSUPPORTED;
  if (!ptr_ok(ws, 256) || ws_bytes < pararnn_lm_layer_norm_vjp_workspace_bytes(N, D)) return PARARNN_ERR_WORKSPACE;
  const bool params = d_weight || d_bias;
  const int64_t groups = grad_groups(N, D);
  const NormGradArgs a{dy, s, d_sum, weight, stats, d_x, dy_stride, s_stride, d_sum_stride, d_x_stride, N, D,
                       params ? static_cast<float*>(ws) : nullptr};
  hipStream_t st = static_cast<hipStream_t>(stream);
  const auto run = [&](auto t) {
    using T = decltype(t);
    shape_of<T>(D, [&](auto sh) { k_norm_grad<T, decltype(sh)><<<static_cast<unsigned>(groups), grad_threads(decltype(sh)::LPR), 0, st>>>(a); });
  };
  if (N > 0) {
    if (dtype == PARARNN_BF16) run(bf16{});
    else run(float{});
  }
  if (params)
    k_norm_params<<<static_cast<unsigned>(ceil_div(2 * D, WAVE)), 1024, 0, st>>>(a.part, groups, D, d_weight, d_bias);
  return launched();
}
