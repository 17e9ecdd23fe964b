// lm_logp.hip -- log probabilities of given tokens, entropy and top alternatives of pararnn_lm.h, and their gradient.

#include "lm_common.h"

namespace lm {

constexpr int NT = 256;

// combines v over the workgroup with f, the same result for every thread
template <class V, class F>
DEV V block_fold(V v, V (&sh)[NT / WAVE], F f) {
#pragma unroll
  for (int o = WAVE / 2; o > 0; o >>= 1) v = f(v, __shfl_xor(v, o, WAVE));
  __syncthreads();
  if (threadIdx.x % WAVE == 0) sh[threadIdx.x / WAVE] = v;
  __syncthreads();
  v = sh[0];
#pragma unroll
  for (int w = 1; w < NT / WAVE; ++w) v = f(v, sh[w]);
  return v;
}

// A logit and its index as one whole number that orders by (value descending, index ascending) as a larger number
// first: the value's bits in the order of the values (-0 counts as 0, NaN as -infinity), the index complemented.
DEV uint64_t rank_key(float z, uint32_t index) {
  const float v = z != z ? -INFINITY : z + 0.0f;
  const uint32_t b = __float_as_uint(v);
  const uint32_t o = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
  return (static_cast<uint64_t>(o) << 32) | static_cast<uint32_t>(~index);
}

DEV int64_t target_of(const void* t, int bytes, int64_t n) {
  return bytes == 8 ? static_cast<const int64_t*>(t)[n] : static_cast<const int32_t*>(t)[n];
}

struct LogpArgs {
  const void* z;
  int64_t stride, V;
  const void* targets;
  int tbytes, top;
  float *lse, *logp, *entropy, *top_logp;
  int64_t* top_ids;
};

// one row a workgroup: the maximum, then sum e^{z-m} and sum e^{z-m}(z-m), then one pass for each alternative
template <typename T>
__global__ __launch_bounds__(NT) void k_logp(const LogpArgs p) {
  __shared__ float sh[NT / WAVE];
  __shared__ uint64_t shk[NT / WAVE];
  const int64_t n = blockIdx.x;
  const T* z = static_cast<const T*>(p.z) + n * p.stride;
  float m = -INFINITY;
  for (int64_t j = threadIdx.x; j < p.V; j += NT) m = fmaxf(m, to_f32(z[j]));
  m = block_fold(m, sh, [](float a, float b) { return fmaxf(a, b); });
  const float base = m == -INFINITY ? 0.0f : m;   // nothing left: every term is 0
  float s = 0.0f, e = 0.0f;
  for (int64_t j = threadIdx.x; j < p.V; j += NT) {
    const float t = to_f32(z[j]) - base, w = hw_exp2(kLog2e * t);
    s += w;
    e = fmaf(w, fmaxf(t, -1e30f), e);             // a ruled out token adds 0, not 0 * infinity
  }
  const auto add = [](float a, float b) { return a + b; };
  s = block_fold(s, sh, add);
  e = block_fold(e, sh, add);
  const bool none = s == 0.0f;
  const float ls = kLn2 * hw_log2(s);
  if (threadIdx.x == 0) {
    if (p.lse) p.lse[n] = none ? -INFINITY : m + ls;
    if (p.entropy) p.entropy[n] = none ? 0.0f : ls - e / s;
    if (p.logp) {
      const int64_t t = target_of(p.targets, p.tbytes, n);
      p.logp[n] = t < 0 ? 0.0f : t >= p.V ? NAN : none ? -INFINITY : (to_f32(z[t]) - m) - ls;
    }
  }
  uint64_t last = ~UINT64_C(0);
  for (int k = 0; k < p.top; ++k) {
    uint64_t best = 0;
    for (int64_t j = threadIdx.x; j < p.V; j += NT) {
      const uint64_t key = rank_key(to_f32(z[j]), static_cast<uint32_t>(j));
      if (key < last && key > best) best = key;
    }
    last = block_fold(best, shk, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
    if (threadIdx.x == 0) {
      const int64_t j = static_cast<uint32_t>(~static_cast<uint32_t>(last));
      p.top_ids[n * p.top + k] = j;
      p.top_logp[n * p.top + k] = none ? -INFINITY : (to_f32(z[j]) - m) - ls;
    }
  }
}

struct LogpGradArgs {
  const void* z;
  int64_t stride, V;
  const void* targets;
  int tbytes;
  const float *lse, *entropy, *g_logp, *g_entropy;
  void* dz;
  int64_t dstride;
};

template <typename T>
__global__ __launch_bounds__(NT) void k_logp_grad(const LogpGradArgs p) {
  const int64_t n = blockIdx.x;
  const T* z = static_cast<const T*>(p.z) + n * p.stride;
  T* dz = static_cast<T*>(p.dz) + n * p.dstride;
  const int64_t t = p.targets ? target_of(p.targets, p.tbytes, n) : -1;
  const float lse = p.lse[n], g = t < 0 ? 0.0f : t >= p.V ? NAN : p.g_logp[n];
  const float ge = p.g_entropy ? p.g_entropy[n] : 0.0f, h = p.g_entropy ? p.entropy[n] : 0.0f;
  const bool none = lse == -INFINITY;
  for (int64_t j = threadIdx.x; j < p.V; j += NT) {
    const float l = none ? -INFINITY : to_f32(z[j]) - lse;
    const float q = hw_exp2(kLog2e * l);
    float v = -q * fmaf(ge, fmaxf(l, -1e30f) + h, g);
    if (j == t && !none) v += g;
    dz[j] = from_f32<T>(v);
  }
}

}  // namespace lm

using namespace lm;

extern "C" size_t pararnn_lm_token_logprobs_workspace_bytes(int64_t N, int64_t V, int top) {
  if (!sizes_fit(N, V) || V > INT32_MAX || top < 0 || top > PARARNN_LM_MAX_TOP || top > V) return 0;
  return 256;
}

static pararnn_status check_logp(int dtype, int64_t N, int64_t V, const void* logits, int64_t stride, const void* targets,
                                 int target_bytes) {
  if (!dtype_ok(dtype) || !sizes_fit(N, V) || V > INT32_MAX) return PARARNN_ERR_INVALID_ARG;
  if (targets && target_bytes != 4 && target_bytes != 8) return PARARNN_ERR_INVALID_ARG;
  if (targets && !aligned(targets, static_cast<size_t>(target_bytes))) return PARARNN_ERR_INVALID_ARG;
  if (N > 0 && V > 0 && !ptr_ok(logits, dtype_size(dtype))) return PARARNN_ERR_INVALID_ARG;
  if (!plane_ok(N, stride)) return PARARNN_ERR_INVALID_ARG;
  if (N > kMaxGrid) return PARARNN_ERR_UNSUPPORTED;
  return PARARNN_OK;
}

extern "C" pararnn_status pararnn_lm_token_logprobs(int dtype, int64_t N, int64_t V, const void* logits, int64_t stride,
                                                    const void* targets, int target_bytes, float* lse, float* logp,
                                                    float* entropy, int top, float* top_logp, int64_t* top_ids,
                                                    void* ws, size_t ws_bytes, void* stream) {
  if (const pararnn_status st = check_logp(dtype, N, V, logits, stride, targets, target_bytes)) return st;
  if (top < 0 || top > PARARNN_LM_MAX_TOP || top > V) return PARARNN_ERR_INVALID_ARG;
  if (N == 0) return PARARNN_OK;
  if (!ptr_ok(lse, 4, false) || !ptr_ok(logp, 4, targets != nullptr) || (logp && !targets) || !ptr_ok(entropy, 4, false) ||
      !ptr_ok(top_logp, 4, top > 0) || !ptr_ok(top_ids, 8, top > 0))
    return PARARNN_ERR_INVALID_ARG;
  if (!ptr_ok(ws, 256) || ws_bytes < pararnn_lm_token_logprobs_workspace_bytes(N, V, top)) return PARARNN_ERR_WORKSPACE;
  const LogpArgs a{logits, stride, V, targets, target_bytes, top, lse, logp, entropy, top_logp, top_ids};
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (dtype == PARARNN_BF16) k_logp<bf16><<<static_cast<unsigned>(N), NT, 0, st>>>(a);
  else k_logp<float><<<static_cast<unsigned>(N), NT, 0, st>>>(a);
  return launched();
}

extern "C" pararnn_status pararnn_lm_token_logprobs_vjp(int dtype, int64_t N, int64_t V, const void* logits, int64_t stride,
                                                        const void* targets, int target_bytes, const float* lse,
                                                        const float* entropy, const float* g_logp, const float* g_entropy,
                                                        void* d_logits, int64_t d_stride, void* stream) {
  if (const pararnn_status st = check_logp(dtype, N, V, logits, stride, targets, target_bytes)) return st;
  if (N == 0 || V == 0) return PARARNN_OK;
  if (!ptr_ok(lse, 4) || !ptr_ok(g_logp, 4, targets != nullptr) || !ptr_ok(g_entropy, 4, false) ||
      !ptr_ok(entropy, 4, g_entropy != nullptr) || !ptr_ok(d_logits, dtype_size(dtype)) || !plane_ok(N, d_stride))
    return PARARNN_ERR_INVALID_ARG;
  const LogpGradArgs a{logits, stride, V, targets, target_bytes, lse, entropy, g_logp, g_entropy, d_logits, d_stride};
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (dtype == PARARNN_BF16) k_logp_grad<bf16><<<static_cast<unsigned>(N), NT, 0, st>>>(a);
  else k_logp_grad<float><<<static_cast<unsigned>(N), NT, 0, st>>>(a);
  return launched();
}
