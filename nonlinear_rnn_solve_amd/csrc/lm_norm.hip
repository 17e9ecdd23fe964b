// lm_norm.hip -- layer normalisation of pararnn_lm.h and its gradients.

#include "lm_common.h"

namespace lm {

constexpr int NT = 256;

// the workgroup's sum of v, the same for every thread: lanes by a butterfly, then the waves in order
DEV float block_sum(float v, float (&sh)[NT / WAVE]) {
#pragma unroll
  for (int o = WAVE / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, WAVE);
  __syncthreads();
  if (threadIdx.x % WAVE == 0) sh[threadIdx.x / WAVE] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < NT / WAVE; ++w) s += sh[w];
  return s;
}

struct NormArgs {
  const void *x, *res;
  const float *weight, *bias;
  void *y, *sum;
  float* stats;
  int64_t sx, sres, sy, ssum, D;
  float eps;
};

// one row a workgroup: the row is read once for the mean, once for the variance about it, once to write
template <typename T>
__global__ __launch_bounds__(NT) void k_norm(const NormArgs p) {
  __shared__ float sh[NT / WAVE];
  const int64_t n = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + n * p.sx;
  const T* res = p.res ? static_cast<const T*>(p.res) + n * p.sres : nullptr;
  T* y = static_cast<T*>(p.y) + n * p.sy;
  T* sum = p.sum ? static_cast<T*>(p.sum) + n * p.ssum : nullptr;
  float s = 0.0f;
  for (int64_t d = threadIdx.x; d < p.D; d += NT) {
    float v = to_f32(x[d]);
    if (res) {
      const T t = from_f32<T>(v + to_f32(res[d]));
      sum[d] = t;
      v = to_f32(t);
    }
    s += v;
  }
  const T* in = res ? sum : x;   // each thread reads back what it wrote itself
  const float mean = block_sum(s, sh) / static_cast<float>(p.D);
  s = 0.0f;
  for (int64_t d = threadIdx.x; d < p.D; d += NT) {
    const float v = to_f32(in[d]) - mean;
    s = fmaf(v, v, s);
  }
  const float rstd = 1.0f / sqrtf(block_sum(s, sh) / static_cast<float>(p.D) + p.eps);
  for (int64_t d = threadIdx.x; d < p.D; d += NT)
    y[d] = from_f32<T>(fmaf((to_f32(in[d]) - mean) * rstd, p.weight[d], p.bias ? p.bias[d] : 0.0f));
  if (p.stats && threadIdx.x == 0) {
    p.stats[2 * n] = mean;
    p.stats[2 * n + 1] = rstd;
  }
}

struct NormGradArgs {
  const void *dy, *s, *dsum;
  const float *weight, *stats;
  void* dx;
  int64_t sdy, ss, sdsum, sdx, N, D;
  float *dweight, *dbias;
};

template <typename T>
__global__ __launch_bounds__(NT) void k_norm_dx(const NormGradArgs p) {
  __shared__ float sh[NT / WAVE];
  const int64_t n = blockIdx.x;
  const T* dy = static_cast<const T*>(p.dy) + n * p.sdy;
  const T* s = static_cast<const T*>(p.s) + n * p.ss;
  const T* dsum = p.dsum ? static_cast<const T*>(p.dsum) + n * p.sdsum : nullptr;
  T* dx = static_cast<T*>(p.dx) + n * p.sdx;
  const float mean = p.stats[2 * n], rstd = p.stats[2 * n + 1];
  float c1 = 0.0f, c2 = 0.0f;
  for (int64_t d = threadIdx.x; d < p.D; d += NT) {
    const float g = to_f32(dy[d]) * p.weight[d];
    c1 += g;
    c2 = fmaf(g, (to_f32(s[d]) - mean) * rstd, c2);
  }
  c1 = block_sum(c1, sh) / static_cast<float>(p.D);
  c2 = block_sum(c2, sh) / static_cast<float>(p.D);
  for (int64_t d = threadIdx.x; d < p.D; d += NT) {
    const float g = to_f32(dy[d]) * p.weight[d], xn = (to_f32(s[d]) - mean) * rstd;
    float v = rstd * (g - c1 - xn * c2);
    if (dsum) v += to_f32(dsum[d]);
    dx[d] = from_f32<T>(v);
  }
}

// parameter sums, a column a thread, rows in ascending order (launched before k_norm_dx, which may write over dy)
template <typename T>
__global__ __launch_bounds__(WAVE) void k_norm_params(const NormGradArgs p) {
  const int64_t d = static_cast<int64_t>(blockIdx.x) * WAVE + threadIdx.x;
  if (d >= p.D) return;
  float sw = 0.0f, sb = 0.0f;
  for (int64_t n = 0; n < p.N; ++n) {
    const float dy = to_f32(static_cast<const T*>(p.dy)[n * p.sdy + d]);
    const float xn = (to_f32(static_cast<const T*>(p.s)[n * p.ss + d]) - p.stats[2 * n]) * p.stats[2 * n + 1];
    sw = fmaf(dy, xn, sw);
    sb += dy;
  }
  if (p.dweight) p.dweight[d] = sw;
  if (p.dbias) p.dbias[d] = sb;
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
  if (D > PARARNN_LM_NORM_MAX_D || N > kMaxGrid) return PARARNN_ERR_UNSUPPORTED;
  const NormArgs a{x, residual, weight, bias, y, sum, stats, x_stride, residual_stride, y_stride, sum_stride, D, eps};
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (dtype == PARARNN_BF16) k_norm<bf16><<<static_cast<unsigned>(N), NT, 0, st>>>(a);
  else k_norm<float><<<static_cast<unsigned>(N), NT, 0, st>>>(a);
  return launched();
}

extern "C" size_t pararnn_lm_layer_norm_vjp_workspace_bytes(int64_t N, int64_t D) {
  return sizes_fit(N, D) ? 256 : 0;
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
  if (D > PARARNN_LM_NORM_MAX_D || N > kMaxGrid) return PARARNN_ERR_UNSUPPORTED;
  if (!ptr_ok(ws, 256) || ws_bytes < pararnn_lm_layer_norm_vjp_workspace_bytes(N, D)) return PARARNN_ERR_WORKSPACE;
  const NormGradArgs a{dy, s, d_sum, weight, stats, d_x, dy_stride, s_stride, d_sum_stride, d_x_stride, N, D, d_weight, d_bias};
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (d_weight || d_bias) {
    const unsigned g = static_cast<unsigned>(ceil_div(D, WAVE));
    if (dtype == PARARNN_BF16) k_norm_params<bf16><<<g, WAVE, 0, st>>>(a);
    else k_norm_params<float><<<g, WAVE, 0, st>>>(a);
  }
  if (N > 0) {
    if (dtype == PARARNN_BF16) k_norm_dx<bf16><<<static_cast<unsigned>(N), NT, 0, st>>>(a);
    else k_norm_dx<float><<<static_cast<unsigned>(N), NT, 0, st>>>(a);
  }
  return launched();
}
