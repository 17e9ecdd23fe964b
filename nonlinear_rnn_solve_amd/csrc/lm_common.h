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
// v_exp_f32 is 2^x, v_log_f32 log2, v_rcp_f32 1/x, each about 1 ulp
DEV float hw_exp2(float x) { return __builtin_amdgcn_exp2f(x); }
DEV float hw_log2(float x) { return __builtin_amdgcn_logf(x); }
DEV float hw_rcp(float x) { return __builtin_amdgcn_rcpf(x); }
DEV float sigmoid(float x) { return hw_rcp(1.0f + hw_exp2(-kLog2e * x)); }

// softplus(x) = max(x, 0) + log1p(e^-|x|); log1p(e) = log(w) e / (w - 1) with w = fl(1 + e), exact in the
// rounding of w (W. Kahan's correction), since small rates (1e-4 and below) set the longest memories
DEV float softplus(float x) {
  const float e = hw_exp2(-kLog2e * fabsf(x));
  const float w = 1.0f + e;
  const float l = w == 1.0f ? e : kLn2 * hw_log2(w) * e * hw_rcp(w - 1.0f);
  return fmaxf(x, 0.0f) + l;
}

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

// V consecutive elements in their storage type, loaded as one access of 2 to 16 bytes and kept as 32-bit words (two
// bf16 a word: element by element the compiler would spend a register on each)
template <typename T, int V> struct Vec {
  static constexpr int N = V * sizeof(T) < 4 ? 1 : V * static_cast<int>(sizeof(T)) / 4;
  uint32_t w[N];
  DEV float get(int v) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[v]);
    else if constexpr (V == 1) return __uint_as_float(w[0] << 16);
    else return __uint_as_float(v % 2 ? w[v / 2] & 0xffff0000u : w[v / 2] << 16);
  }
};
template <typename T, int V> DEV Vec<T, V> pack_vec(const float (&x)[V]) {
  Vec<T, V> r;
#pragma unroll
  for (int k = 0; k < Vec<T, V>::N; ++k) {
    if constexpr (sizeof(T) == 4) r.w[k] = __float_as_uint(x[k]);
    else if constexpr (V == 1) r.w[k] = bf16_bits(x[0]);
    else r.w[k] = bf16_bits(x[2 * k]) | static_cast<uint32_t>(bf16_bits(x[2 * k + 1])) << 16;
  }
  return r;
}

// The first `n` of V elements at p (all of them where n >= V), as one access at any alignment of the element: the GPU
// runs in unaligned access mode, so odd row lengths need no narrower loads.  The elements past n are `fill`.  LAST: nothing
// reads them after this kernel, so they need not stay in the caches (the logits in their gradient: 257 against 280 us for
// the pass over 4096 x 32000 float32, 23.3 against 22.7 for 65536 x 256 bfloat16).
template <typename T, int V> using LooseWords __attribute__((aligned(sizeof(T)))) =
    uint32_t __attribute__((ext_vector_type(Vec<T, V>::N)));
template <typename T, int V, bool LAST = false> DEV Vec<T, V> load_row(const T* p, int64_t n, T fill) {
  static_assert(V * sizeof(T) >= 4, "whole words");
  Vec<T, V> r;
  if (n >= V) {
    const auto* s = reinterpret_cast<const LooseWords<T, V>*>(p);
    const LooseWords<T, V> q = LAST ? __builtin_nontemporal_load(s) : *s;
#pragma unroll
    for (int k = 0; k < Vec<T, V>::N; ++k) r.w[k] = q[k];
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const T e = v < n ? p[v] : fill;
      if constexpr (sizeof(T) == 4) r.w[v] = __float_as_uint(e);
      else r.w[v / 2] = v % 2 ? r.w[v / 2] | static_cast<uint32_t>(e.u) << 16 : e.u;
    }
  }
  return r;
}
// Stores do not stay in the caches: what is written once should not push out what is read, and the lines need not be
// fetched first (layer norm's training pass, float32 5001 x 2047: 43.6 against 52.5 us; log probabilities', 4096 x 32000:
// 273 against 299 us).
template <typename T, int V> DEV void store_row(T* p, int64_t n, const float (&x)[V]) {
  const Vec<T, V> r = pack_vec<T, V>(x);
  if (n >= V) {
    LooseWords<T, V> q;
#pragma unroll
    for (int k = 0; k < Vec<T, V>::N; ++k) q[k] = r.w[k];
    __builtin_nontemporal_store(q, reinterpret_cast<LooseWords<T, V>*>(p));
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v < n) p[v] = from_f32<T>(x[v]);
  }
}

// Sums over 16 consecutive lanes (a DPP row), over a wave: the same value for every lane, in a fixed order.
template <int CTRL> DEV float dpp(float v) {
  return __uint_as_float(static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(0, static_cast<int>(__float_as_uint(v)), CTRL, 0xf, 0xf, true)));
}
DEV float row_sum(float v) {
  v += dpp<0xb1>(v);    // quad_perm [1,0,3,2]
  v += dpp<0x4e>(v);    // quad_perm [2,3,0,1]
  v += dpp<0x141>(v);   // row_half_mirror
  v += dpp<0x140>(v);   // row_mirror
  return v;
}
DEV float read_lane(float v, int lane) {
  return __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(__float_as_uint(v)), lane)));
}
DEV float wave_sum(float v) {
  v = row_sum(v);
  return (read_lane(v, 0) + read_lane(v, 16)) + (read_lane(v, 32) + read_lane(v, 48));
}

// the maximum over 16 consecutive lanes, over a wave (a NaN loses)
DEV float row_max(float v) {
  v = fmaxf(v, dpp<0xb1>(v));
  v = fmaxf(v, dpp<0x4e>(v));
  v = fmaxf(v, dpp<0x141>(v));
  v = fmaxf(v, dpp<0x140>(v));
  return v;
}
DEV float wave_max(float v) {
  v = row_max(v);
  return fmaxf(fmaxf(read_lane(v, 0), read_lane(v, 16)), fmaxf(read_lane(v, 32), read_lane(v, 48)));
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
inline int64_t ceil_div(int64_t a, int64_t b) { return a / b + (a % b != 0); }   // a >= 0 of any size
// a launch has fewer than 2^32 threads
inline bool grid_ok(int64_t blocks, int64_t threads) { return blocks <= INT64_C(0xffffffff) / threads; }

}  // namespace lm
#endif
