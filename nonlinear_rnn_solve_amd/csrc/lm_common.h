// lm_common.h -- what the kernels of libpararnn_lm.so share: element loads and stores of the two storage
// types, wave and workgroup sums in a fixed order, argument checks of the C entries.
#ifndef PARARNN_LM_COMMON_H
#define PARARNN_LM_COMMON_H

#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstddef>
#include <cstdint>

#include "pararnn_lm.h"

#define DEV __device__ __forceinline__

namespace lm {

constexpr int WAVE = 64;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// v_exp_f32 is 2^x, v_log_f32 log2, v_rcp_f32 1/x, v_rsq_f32 1/sqrt, each about 1 ulp
DEV float hw_exp2(float x) { return __builtin_amdgcn_exp2f(x); }
DEV float hw_log2(float x) { return __builtin_amdgcn_logf(x); }
DEV float hw_rcp(float x) { return __builtin_amdgcn_rcpf(x); }
DEV float hw_rsq(float x) { return __builtin_amdgcn_rsqf(x); }
DEV float sigmoid(float x) { return hw_rcp(1.0f + hw_exp2(-kLog2e * x)); }

struct bf16 { uint16_t u; };   // storage only

DEV float to_f32(float x) { return x; }
DEV float to_f32(bf16 x) { return __uint_as_float(static_cast<uint32_t>(x.u) << 16); }
// bf16 results are rounded once, to the nearest even, by the hardware conversion
DEV uint16_t bf16_bits(float x) {
  const __bf16 h = static_cast<__bf16>(x);
  return __builtin_bit_cast(uint16_t, h);
}
template <typename T> DEV T from_f32(float x);
template <> DEV float from_f32<float>(float x) { return x; }
template <> DEV bf16 from_f32<bf16>(float x) { return bf16{bf16_bits(x)}; }

// V consecutive elements as one load or store of 2 to 16 bytes, and their values
template <typename T, int V> struct alignas(sizeof(T) * V) Vec {
  T e[V];
};
template <typename T, int V> DEV Vec<T, V> load_vec(const T* p) { return *reinterpret_cast<const Vec<T, V>*>(p); }
template <typename T, int V> DEV void store_vec(T* p, const float (&x)[V]) {
  Vec<T, V> v;
#pragma unroll
  for (int k = 0; k < V; ++k) v.e[k] = from_f32<T>(x[k]);
  *reinterpret_cast<Vec<T, V>*>(p) = v;
}

// ---------------- host: argument checks ----------------
inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline bool dtype_ok(int dt) { return dt == PARARNN_F32 || dt == PARARNN_BF16; }
inline size_t dtype_size(int dt) { return dt == PARARNN_BF16 ? 2 : 4; }
// a required (or, with `need` false, optional) pointer at the alignment of its element type
inline bool ptr_ok(const void* p, size_t align, bool need = true) { return p ? aligned(p, align) : !need; }
// the product of nonnegative sizes, times 16 bytes, fits int64
inline bool sizes_fit(int64_t a, int64_t b, int64_t c = 1) {
  if (a < 0 || b < 0 || c < 0) return false;
  if (a == 0 || b == 0 || c == 0) return true;
  const int64_t lim = INT64_MAX / 16;
  if (a > lim / b) return false;
  return c <= lim / (a * b);
}
// the last element of a plane of n rows with stride s and d dense elements has an offset that fits int64
inline bool plane_ok(int64_t n, int64_t s) { return s >= 0 && (n <= 1 || s <= INT64_MAX / 16 / (n - 1)); }
inline pararnn_status launched() { return hipGetLastError() == hipSuccess ? PARARNN_OK : PARARNN_ERR_HIP; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
constexpr int64_t kMaxGrid = INT64_C(0x7fffffff);

}  // namespace lm
#endif
