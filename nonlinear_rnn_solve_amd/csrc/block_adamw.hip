// block_adamw.hip -- one AdamW step over many tensors, with moments in 32 or in 8 bits (pararnn_block.h).

#include "block_common.h"

namespace lm {

// The tensors of one launch stand in its arguments, so that nothing is copied to the device before it and gradients may move from
// step to step; a workgroup finds its tensor among them by its number.  A lane holds V consecutive elements of P pieces, all
// of whose loads are in flight before the first is used.  A piece of a wave is one block of the 8-bit moments.
constexpr int V = 4, P = 4, PIECE = WAVE * V, CHUNK = 4 * P * PIECE;   // elements of a workgroup of four waves
constexpr int TENSORS = 64;
static_assert(PIECE == PARARNN_BLOCK_ADAMW_BLOCK, "a wave's piece is a block");

struct AdamwTensor {
  void* param;
  const void* grad;
  int64_t numel, offset;
};
struct AdamwArgs {
  AdamwTensor t[TENSORS];
  uint32_t first[TENSORS + 1];  // first workgroup of each tensor
  int32_t count;
  float beta1, beta2, rest1, rest2, eps, decay, lr, grad_scale;
  float c1, c2;                 // 1 / (1 - beta1^step), 1 / sqrt(1 - beta2^step)
  double b1, b2;
  int64_t step;
  const float *lr_ptr, *grad_scale_ptr;
  const int64_t* step_ptr;
  uint64_t seed;
  void *m, *v;
  float *m_scale, *v_scale;
};
static_assert(sizeof(AdamwArgs) <= 4096, "kernel arguments");

__host__ DEV double power(double b, int64_t n) {
  double r = 1.0;
  for (; n > 0; n >>= 1, b *= b)
    if (n & 1) r *= b;
  return r;
}

// C. Wellons's 32-bit mixer (a bijection found by searching for the least bias)
DEV uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7feb352du;
  x ^= x >> 15;
  x *= 0x846ca68bu;
  return x ^ x >> 16;
}

// 8-bit codes: BIAS 15 with a sign (m), BIAS 31 without (v).  A code's exponent and fraction in a float's top bits are the value
// times 2^(BIAS - 127): the smallest codes are that float's denormal ones, which products keep.
template <int BIAS> DEV float decode(uint32_t code, float scale) {
  const uint32_t magnitude = BIAS == 15 ? code & 127 : code;
  float x = __uint_as_float(magnitude << 20) * __uint_as_float(static_cast<uint32_t>(127 + 127 - BIAS) << 23) * scale;
  if constexpr (BIAS == 15) x = __uint_as_float(__float_as_uint(x) | (code & 128) << 24);
  return x;
}
// of |x| <= 1.875 2^e, rounded up where its place between two codes and `number` / 2^20 add up to one or more (a number less by one:
// to more than one)
template <int BIAS> DEV uint32_t encode(float x, int e, uint32_t number) {
  const float y = ldexpf(fabsf(x), -e);
  const uint32_t normal = ((__float_as_uint(y) + number) >> 20) - (127 - BIAS) * 8;
  const uint32_t small = (static_cast<uint32_t>(ldexpf(y, BIAS + 22)) + number) >> 20;
  const uint32_t code = y < __uint_as_float(static_cast<uint32_t>(128 - BIAS) << 23) ? small : normal;
  return BIAS == 15 && x < 0.0f ? code | 128 : code;
}
// the exponent of the smallest power of two of at least 2^-80 whose 1.875-fold is not below `most`
DEV int scale_exponent(float most) {
  const uint32_t u = __float_as_uint(most);
  const int e = static_cast<int>(u >> 23) - 127 + ((u & 0x7fffffu) > 0x700000u);
  return e > -80 ? e : -80;
}
DEV float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

template <typename W> using Loose = W __attribute__((aligned(1)));
DEV uint32_t load_codes(const void* p, int64_t at) {
  return *reinterpret_cast<const Loose<uint32_t>*>(static_cast<const uint8_t*>(p) + at);
}

struct Rates {
  float decay, rate, c2, grad_scale;   // decay: lr weight_decay
};

// What a step takes from p is summed by itself: 1 - lr weight_decay would be rounded to a multiple of 2^-24, a decay of 1e-7 to 1.2e-7
// and one below 3e-8 to nothing, for all parameters and steps alike.  (An infinite p would be taken from itself.)
DEV float new_param(const AdamwArgs& a, const Rates& r, float p, float m, float v) {
  const float step = (r.rate * m) / fmaf(sqrtf(v), r.c2, a.eps);
  return p - (fabsf(p) < __builtin_huge_valf() ? fmaf(p, r.decay, step) : step);
}

// PT, GT: types of parameters and gradients.  Bound by memory: 28 bytes an element with float32 and 32-bit moments, 12 to 16
// with 8 bits.  116 million float32 parameters: 595 us (5.5 TB/s; a large copy runs at 5.06); with bfloat16 gradients and 8-bit
// moments 335 to 345 (14 bytes, 4.8 TB/s).
template <typename PT, typename GT, bool EIGHT>
__global__ __launch_bounds__(256) void k_adamw(const AdamwArgs a) {
  int j = 0;
  for (int s = TENSORS / 2; s; s /= 2)
    if (j + s < a.count && a.first[j + s] <= blockIdx.x) j += s;
  const AdamwTensor t = a.t[j];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t base = static_cast<int64_t>(blockIdx.x - a.first[j]) * CHUNK + wave * (P * PIECE) + lane * V;

  PT* param = static_cast<PT*>(t.param) + base;
  const GT* grad = static_cast<const GT*>(t.grad) + base;
  const int64_t left = t.numel - base, at = t.offset + base;
  Vec<PT, V> p[P];
  Vec<GT, V> g[P];
  Vec<float, V> m[P], v[P];
  uint32_t mc[P], vc[P];
  float ms[P], vs[P];
#pragma unroll
  for (int k = 0; k < P; ++k) {
    const int64_t n = left - k * PIECE;
    p[k] = load_row<PT, V>(param + k * PIECE, n, PT{});
    g[k] = load_row<GT, V, true>(grad + k * PIECE, n, GT{});
    if constexpr (EIGHT) {
      // a wave's piece that has any element of the tensor is wholly inside the state
      const bool any = n + lane * V > 0;
      const int64_t block = (at + k * PIECE) / PIECE;
      mc[k] = any ? load_codes(a.m, at + k * PIECE) : 0;
      vc[k] = any ? load_codes(a.v, at + k * PIECE) : 0;
      ms[k] = any ? a.m_scale[block] : 0.0f;
      vs[k] = any ? a.v_scale[block] : 0.0f;
    } else {
      m[k] = load_row<float, V>(static_cast<const float*>(a.m) + at + k * PIECE, n, 0.0f);
      v[k] = load_row<float, V>(static_cast<const float*>(a.v) + at + k * PIECE, n, 0.0f);
    }
  }

  const float lr = a.lr_ptr ? *a.lr_ptr : a.lr;
  int64_t step = a.step;
  float c1 = a.c1, c2 = a.c2;
  if (a.step_ptr) {
    step = *a.step_ptr;
    c1 = static_cast<float>(1.0 / (1.0 - power(a.b1, step)));
    c2 = static_cast<float>(1.0 / sqrt(1.0 - power(a.b2, step)));
  }
  const Rates r{lr * a.decay, lr * c1, c2, a.grad_scale_ptr ? *a.grad_scale_ptr : a.grad_scale};
  const uint32_t lo = static_cast<uint32_t>(a.seed), hi = static_cast<uint32_t>(a.seed >> 32);
  const uint32_t key = mix(lo ^ mix(hi) ^ mix(static_cast<uint32_t>(step) ^ mix(static_cast<uint32_t>(step >> 32))));

#pragma unroll
  for (int k = 0; k < P; ++k) {
    const int64_t n = left - k * PIECE, place = at + k * PIECE;
    if (n + lane * V <= 0) break;      // uniform: nothing of the tensor is left
    float np[V], nm[V], nv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float x = g[k].get(i) * r.grad_scale;
      const float m0 = EIGHT ? decode<15>(mc[k] >> (8 * i) & 255, ms[k]) : m[k].get(i);
      const float v0 = EIGHT ? decode<31>(vc[k] >> (8 * i) & 255, vs[k]) : v[k].get(i);
      // each product and sum rounded by itself: a moment in 8 bits then depends on no compiler's choice of fused steps, of which one
      // in 400 000 would round it the other way
      const float m1 = a.beta1 * m0, m2 = a.rest1 * x, v1 = a.beta2 * v0, v2 = a.rest2 * x;
      const float v3 = v2 * x;
      nm[i] = m1 + m2;
      nv[i] = v1 + v3;
      np[i] = new_param(a, r, p[k].get(i), nm[i], nv[i]);
    }
    store_row<PT, V>(param + k * PIECE, n, np);
    if constexpr (EIGHT) {
      float mm = 0.0f, mv = 0.0f;
      bool bad = false;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (i >= n) nm[i] = nv[i] = 0.0f;
        mm = fmaxf(mm, fabsf(nm[i]));
        mv = fmaxf(mv, nv[i]);
        bad = bad || !(fabsf(nm[i]) < __builtin_huge_valf()) || !(nv[i] < __builtin_huge_valf());
      }
      bad = __builtin_amdgcn_ballot_w64(bad) != 0;
      const int em = scale_exponent(wave_max(mm)), ev = scale_exponent(wave_max(mv));
      bad = bad || em > 127 || ev > 127;   // no float holds 2^128
      uint32_t cm = 0, cv = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint64_t e = static_cast<uint64_t>(place) + i;
        const uint32_t h = mix(static_cast<uint32_t>(e) ^ mix(key ^ static_cast<uint32_t>(e >> 32)));
        cm |= encode<15>(nm[i], em, (h & 0xffff) << 4) << (8 * i);
        // more than one, for v: a tie goes down, its chance is 2^-16 lower than its place.  Elementary forms that scale by torch's ldexp are
        // short of their ties where that is no power of two on this GPU (131071.99 for 2^17), and v's codes are compared with theirs
        const uint32_t up = (h >> 16) << 4;
        cv |= encode<31>(nv[i], ev, up ? up - 1 : 0) << (8 * i);
      }
      *reinterpret_cast<Loose<uint32_t>*>(static_cast<uint8_t*>(a.m) + place) = bad ? 0 : cm;
      *reinterpret_cast<Loose<uint32_t>*>(static_cast<uint8_t*>(a.v) + place) = bad ? 0 : cv;
      if (lane == 0) {
        a.m_scale[place / PIECE] = bad ? __builtin_nanf("") : power_of_two(em);
        a.v_scale[place / PIECE] = bad ? __builtin_nanf("") : power_of_two(ev);
      }
    } else {
      store_row<float, V>(static_cast<float*>(a.m) + place, n, nm);
      store_row<float, V>(static_cast<float*>(a.v) + place, n, nv);
    }
  }
}

// A thread decodes 8 codes of each moment: 2 bytes in and 4 out an element (116 million: 117 us, 6 TB/s).
__global__ __launch_bounds__(256) void k_adamw_moments(int64_t n, const void* m, const void* v, const float* m_scale,
                                                       const float* v_scale, bf16* m_out, bf16* v_out) {
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (at >= n) return;
  const float ms = m_scale[at / PIECE], vs = v_scale[at / PIECE];
  float x[8], y[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t cm = load_codes(m, at + 4 * h), cv = load_codes(v, at + 4 * h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[4 * h + i] = decode<15>(cm >> (8 * i) & 255, ms);
      y[4 * h + i] = decode<31>(cv >> (8 * i) & 255, vs);
    }
  }
  store_row<bf16, 8>(m_out + at, 8, x);
  store_row<bf16, 8>(v_out + at, 8, y);
}

// ---------------- host ----------------
template <typename PT, typename GT> static void launch(const AdamwArgs& a, bool eight, hipStream_t stream) {
  const dim3 grid(a.first[a.count]);
  if (eight) k_adamw<PT, GT, true><<<grid, dim3(256), 0, stream>>>(a);
  else k_adamw<PT, GT, false><<<grid, dim3(256), 0, stream>>>(a);
}

}  // namespace lm

using namespace lm;

extern "C" pararnn_status pararnn_block_adamw(const pararnn_block_adamw_args* q, const pararnn_block_adamw_tensor* tensors,
                                              int64_t count, void* stream) {
  if (!q || count < 0 || (count > 0 && !tensors) || (q->bits != 8 && q->bits != 32)) return PARARNN_ERR_INVALID_ARG;
  if (!(q->beta1 >= 0 && q->beta1 < 1 && q->beta2 >= 0 && q->beta2 < 1 && q->eps >= 0 && std::isfinite(q->eps) &&
        std::isfinite(q->weight_decay)))
    return PARARNN_ERR_INVALID_ARG;
  if ((!q->lr_ptr && !std::isfinite(q->lr)) || (!q->grad_scale_ptr && !std::isfinite(q->grad_scale)) || (!q->step_ptr && q->step < 1))
    return PARARNN_ERR_INVALID_ARG;
  if (!ptr_ok(q->lr_ptr, 4, false) || !ptr_ok(q->grad_scale_ptr, 4, false) || !ptr_ok(q->step_ptr, 8, false))
    return PARARNN_ERR_INVALID_ARG;
  const bool eight = q->bits == 8;
  bool any = false;
  for (int64_t j = 0; j < count; ++j) {
    const pararnn_block_adamw_tensor& t = tensors[j];
    if (t.numel < 0 || t.offset < 0 || t.offset % PIECE || t.numel > INT64_MAX / 32 || t.offset > INT64_MAX / 32 ||
        !dtype_ok(t.param_dtype) || !dtype_ok(t.grad_dtype) || !ptr_ok(t.param, dtype_size(t.param_dtype), t.numel > 0) ||
        !ptr_ok(t.grad, dtype_size(t.grad_dtype), t.numel > 0))
      return PARARNN_ERR_INVALID_ARG;
    any = any || t.numel > 0;
  }
  if (!ptr_ok(q->m, eight ? 1 : 4, any) || !ptr_ok(q->v, eight ? 1 : 4, any) || !ptr_ok(q->m_scale, 4, any && eight) ||
      !ptr_ok(q->v_scale, 4, any && eight))
    return PARARNN_ERR_INVALID_ARG;
  for (int64_t j = 0; j < count; ++j)
    if (!grid_ok(ceil_div(tensors[j].numel, CHUNK), 256)) return PARARNN_ERR_UNSUPPORTED;

  AdamwArgs a{};
  a.b1 = q->beta1, a.b2 = q->beta2;
  a.beta1 = static_cast<float>(q->beta1), a.beta2 = static_cast<float>(q->beta2);
  a.rest1 = static_cast<float>(1 - q->beta1), a.rest2 = static_cast<float>(1 - q->beta2);
  a.eps = static_cast<float>(q->eps), a.decay = static_cast<float>(q->weight_decay);
  a.lr = static_cast<float>(q->lr), a.grad_scale = static_cast<float>(q->grad_scale);
  a.step = q->step, a.step_ptr = q->step_ptr, a.lr_ptr = q->lr_ptr, a.grad_scale_ptr = q->grad_scale_ptr;
  if (!q->step_ptr) {
    a.c1 = static_cast<float>(1.0 / (1.0 - power(q->beta1, q->step)));
    a.c2 = static_cast<float>(1.0 / std::sqrt(1.0 - power(q->beta2, q->step)));
  }
  a.seed = q->seed;
  a.m = q->m, a.v = q->v, a.m_scale = q->m_scale, a.v_scale = q->v_scale;
  // one launch for each 64 tensors of the same types; those of other types wait for a launch of their own
  const auto st = static_cast<hipStream_t>(stream);
  for (int types = 0; types < 4; ++types) {
    const int pt = types & 1 ? PARARNN_BF16 : PARARNN_F32, gt = types & 2 ? PARARNN_BF16 : PARARNN_F32;
    const auto flush = [&] {
      if (a.count == 0) return PARARNN_OK;
      if (pt == PARARNN_F32) {
        if (gt == PARARNN_F32) launch<float, float>(a, eight, st);
        else launch<float, bf16>(a, eight, st);
      } else {
        if (gt == PARARNN_F32) launch<bf16, float>(a, eight, st);
        else launch<bf16, bf16>(a, eight, st);
      }
      a.count = 0;
      return launched();
    };
    a.count = 0;
    a.first[0] = 0;
    for (int64_t j = 0; j < count; ++j) {
      const pararnn_block_adamw_tensor& t = tensors[j];
      if (t.param_dtype != pt || t.grad_dtype != gt || t.numel == 0) continue;
      const int64_t blocks = ceil_div(t.numel, CHUNK);
      if (a.count == TENSORS || !grid_ok(a.first[a.count] + blocks, 256)) {
        const pararnn_status r = flush();
        if (r != PARARNN_OK) return r;
      }
      a.t[a.count] = {t.param, t.grad, t.numel, t.offset};
      a.first[a.count + 1] = a.first[a.count] + static_cast<uint32_t>(blocks);
      ++a.count;
    }
    const pararnn_status r = flush();
    if (r != PARARNN_OK) return r;
  }
  return PARARNN_OK;
}

extern "C" pararnn_status pararnn_block_adamw_moments(int64_t n, const void* m, const void* v, const float* m_scale,
                                                      const float* v_scale, void* m_out, void* v_out, void* stream) {
  if (n < 0 || n % PIECE || n > INT64_MAX / 32) return PARARNN_ERR_INVALID_ARG;
  if (!ptr_ok(m, 1, n > 0) || !ptr_ok(v, 1, n > 0) || !ptr_ok(m_scale, 4, n > 0) || !ptr_ok(v_scale, 4, n > 0) ||
      !ptr_ok(m_out, 2, n > 0) || !ptr_ok(v_out, 2, n > 0))
    return PARARNN_ERR_INVALID_ARG;
  const int64_t blocks = ceil_div(n, 8 * 256);
  if (!grid_ok(blocks, 256)) return PARARNN_ERR_UNSUPPORTED;
  if (n == 0) return PARARNN_OK;
  k_adamw_moments<<<dim3(static_cast<uint32_t>(blocks)), dim3(256), 0, static_cast<hipStream_t>(stream)>>>(
      n, m, v, m_scale, v_scale, static_cast<bf16*>(m_out), static_cast<bf16*>(v_out));
  return launched();
}
