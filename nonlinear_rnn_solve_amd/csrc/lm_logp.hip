// lm_logp.hip -- log probabilities of given tokens, entropy and top alternatives of pararnn_lm.h, and their gradient.
//
// One pass over the logits each way (two for the gradient of rows whose lse is large).  The forward kernel is bound by vector
// instructions in bfloat16 (11 an element, two of them conversions and one an exponential; 97% of the issue slots at 4096 x
// 131072 with 5 alternatives, 192 us, 5.6 TB/s), by memory in float32 (4096 x 32000: 92 us, 5.7 TB/s), by one CU's instructions
// for few rows (32 x 50001 with 20 alternatives: 11 us), by instructions and the launch's own start and end for short rows
// (bf16 65536 x 256: 10 to 11 us, 46% of the issue slots of the whole launch).  The gradient is bound by memory (4096 x 32000
// float32: 171 us for 1.05 GB, 6.1 TB/s).

#include <algorithm>
#include <type_traits>

#include "lm_common.h"

namespace lm {

// A logit and its index as one whole number that orders by (value descending, index ascending) as a larger number
// first: the value's bits in the order of the values (-0 counts as 0, NaN as -infinity), the index complemented.
DEV uint64_t rank_key(float z, uint32_t index) {
  const float v = z != z ? -INFINITY : z + 0.0f;
  const uint32_t b = __float_as_uint(v);
  const uint32_t o = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
  return (static_cast<uint64_t>(o) << 32) | static_cast<uint32_t>(~index);
}

// the value in a key
DEV float key_value(uint64_t key) {
  const uint32_t o = static_cast<uint32_t>(key >> 32);
  return __uint_as_float(o ^ (o & 0x80000000u ? 0x80000000u : 0xffffffffu));
}

DEV int64_t target_of(const void* t, int bytes, int64_t n) {
  return bytes == 8 ? static_cast<const int64_t*>(t)[n] : static_cast<const int32_t*>(t)[n];
}

struct LogpArgs {
  const void* z;
  int64_t stride, N, V;
  const void* targets;
  int tbytes, top;
  float *lse, *logp, *entropy, *top_logp;
  int64_t* top_ids;
};

// Running statistics of some logits: their maximum m, z = sum e^{x-m} and s = sum e^{x-m} (x-m), so that
// ln sum e^x = m + ln z and the entropy is ln z - s / z.  m = -infinity: no token (left) among them, z = s = 0.
struct Stat { float m, z, s; };
// t = x - m of a ruled out token is -infinity and its e^t 0: the product is 0, not NaN
DEV float weighted(float w, float t, float add) { return fmaf(w, fmaxf(t, -1e30f), add); }
// the same sums about a maximum `to` >= m
DEV void rebase(Stat& a, float to) {
  const float d = a.m - (to == -INFINITY ? 0.0f : to), f = hw_exp2(kLog2e * d);
  a.s = f * weighted(a.z, d, a.s);
  a.z *= f;
  a.m = to;
}

// the statistics of the LPR lanes of a row, joined in a fixed order, for each of them
template <int LPR> DEV void join(Stat& a, float (&sh)[3][LPR > WAVE ? LPR / WAVE : 1]) {
  float m = LPR == 16 ? row_max(a.m) : wave_max(a.m);
  if constexpr (LPR > WAVE) {
    if (threadIdx.x % WAVE == 0) sh[0][threadIdx.x / WAVE] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < LPR / WAVE; ++w) m = fmaxf(m, sh[0][w]);
  }
  rebase(a, m);
  a.z = LPR == 16 ? row_sum(a.z) : wave_sum(a.z);
  a.s = LPR == 16 ? row_sum(a.s) : wave_sum(a.s);
  if constexpr (LPR > WAVE) {
    if (threadIdx.x % WAVE == 0) {
      sh[1][threadIdx.x / WAVE] = a.z;
      sh[2][threadIdx.x / WAVE] = a.s;
    }
    __syncthreads();
    a.z = sh[1][0];
    a.s = sh[2][0];
#pragma unroll
    for (int w = 1; w < LPR / WAVE; ++w) {
      a.z += sh[1][w];
      a.s += sh[2][w];
    }
  }
}

// Top alternatives.  While the row streams by, each lane remembers its best chunk (16 bytes of logits): the first with
// its largest value.  With chunks ranked as (value, chunk) keys, the lanes' bests are folded into 64 columns (lane modulo
// 64); the k-th largest of the 64 is a key that at least k logits of the row reach, so the k alternatives are among the
// logits whose (value, chunk) reaches it, and those lie with the lanes whose own best does: a few dozen lanes, whose
// chunks the workgroup reads again.  What passes goes to a list; its entries' ranks are counted and the first k written.
constexpr int kCols = 64, kList = 512;
template <int LPR> struct TopShared {
  uint64_t best[LPR / WAVE][WAVE];
  uint64_t list[kList];
  uint64_t bar;
  uint32_t lanes[LPR];
  uint32_t n_lanes, n;
};

template <typename T, int LPR>
DEV void top_of(const LogpArgs& p, const T* z, int64_t n, uint64_t best, float m, float ls, bool none, TopShared<LPR>& sh) {
  constexpr int V = 16 / sizeof(T);
  const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE;
  sh.best[wave][lane] = best;
  if (threadIdx.x == 0) sh.n_lanes = sh.n = 0;
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int w = 1; w < LPR / WAVE; ++w) best = max(best, sh.best[w][lane]);
    // 0: a lane without a logit.  Keys are unique otherwise (every chunk has one lane).
    int rank = 0;
#pragma unroll
    for (int j = 0; j < kCols; ++j) {
      const uint64_t o = static_cast<uint64_t>(__builtin_amdgcn_readlane(static_cast<int>(best >> 32), j)) << 32 |
                         static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(best), j));
      rank += o > best;
    }
    const uint64_t kth = __ballot(rank == p.top - 1 && best != 0);   // one lane, or none: fewer than k columns have a logit
    const int at = kth ? __ffsll(static_cast<unsigned long long>(kth)) - 1 : 0;
    const uint64_t bar = static_cast<uint64_t>(__builtin_amdgcn_readlane(static_cast<int>(best >> 32), at)) << 32 |
                         static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(best), at));
    if (lane == 0) sh.bar = kth ? bar : 0;
  }
  __syncthreads();
  const uint64_t bar = sh.bar;
  const float reach = bar ? key_value(bar) : -INFINITY;
  if (sh.best[wave][lane] >= bar && sh.best[wave][lane] != 0) sh.lanes[atomicAdd(&sh.n_lanes, 1u)] = threadIdx.x;
  __syncthreads();
  // below 2^31 logits: 32-bit indices throughout
  const uint32_t chunks = static_cast<uint32_t>((p.V + V - 1) / V), rounds = (chunks + LPR - 1) / LPR, lanes = sh.n_lanes;
  for (uint32_t w = threadIdx.x; w < rounds * lanes; w += LPR) {
    const uint32_t q = w / lanes;
    const int64_t c = static_cast<int64_t>(q) * LPR + sh.lanes[w - q * lanes];
    if (c >= chunks) continue;
    const Vec<T, V> x = load_row<T, V>(z + c * V, p.V - c * V, from_f32<T>(-INFINITY));
    float most = -INFINITY;
#pragma unroll
    for (int e = 0; e < V; ++e) most = fmaxf(most, x.get(e));
    if (most < reach) continue;   // most chunks of these lanes
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (c * V + e >= p.V || rank_key(x.get(e), static_cast<uint32_t>(c)) < bar) continue;
      const uint32_t at = atomicAdd(&sh.n, 1u);
      if (at < kList) sh.list[at] = rank_key(x.get(e), static_cast<uint32_t>(c * V + e));
    }
  }
  __syncthreads();
  const auto put = [&](int k, uint64_t key) {
    p.top_ids[n * p.top + k] = static_cast<uint32_t>(~static_cast<uint32_t>(key));
    p.top_logp[n * p.top + k] = none ? -INFINITY : (key_value(key) - m) - ls;   // a row with a NaN has a NaN ls
  };
  const uint32_t count = sh.n;
  if (count <= kList) {
    for (uint32_t i = threadIdx.x; i < count; i += LPR) {
      const uint64_t key = sh.list[i];
      int rank = 0;
      for (uint32_t j = 0; j < count; j += 8) {
        uint64_t o[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) o[u] = sh.list[j + u];   // kList is a multiple of 8
#pragma unroll
        for (int u = 0; u < 8; ++u) rank += j + u < count && o[u] > key;
      }
      if (rank < p.top) put(rank, key);
    }
    return;
  }
  // a row whose large logits fill fewer than k columns overflows the list: a pass over the row for each alternative
  uint64_t last = ~UINT64_C(0);
  for (int k = 0; k < p.top; ++k) {
    uint64_t next = 0;
    for (int64_t j = threadIdx.x; j < p.V; j += LPR) {
      const uint64_t key = rank_key(to_f32(z[j]), static_cast<uint32_t>(j));
      if (key < last && key > next) next = key;
    }
    __syncthreads();
#pragma unroll
    for (int o = WAVE / 2; o > 0; o >>= 1) next = max(next, static_cast<uint64_t>(__shfl_xor(static_cast<unsigned long long>(next), o, WAVE)));
    if (lane == 0) sh.best[wave][0] = next;
    __syncthreads();
    last = sh.best[0][0];
#pragma unroll
    for (int w = 1; w < LPR / WAVE; ++w) last = max(last, sh.best[w][0]);
    if (threadIdx.x == 0) put(k, last);
  }
}

// A row is read once by LPR lanes, chunk by chunk, kAhead chunks of a lane at a time.  With 1024 lanes 64 registers keep
// two workgroups on a CU: 65 cost 306 against 231 us for 4096 x 131072 bf16 (kAhead = 8, which needs more: 298).
constexpr int kAhead = 4;
template <typename T, int LPR, bool TOP>
__global__ __launch_bounds__(LPR > WAVE ? LPR : WAVE) __attribute__((amdgpu_waves_per_eu(LPR > 256 ? 8 : 1)))
void k_logp(const LogpArgs p) {
  constexpr int V = 16 / sizeof(T), NT = LPR > WAVE ? LPR : WAVE;
  __shared__ float sh[3][LPR > WAVE ? LPR / WAVE : 1];
  const int lane = threadIdx.x % LPR;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * (NT / LPR) + threadIdx.x / LPR;
  const bool on = NT == LPR || n < p.N;
  const T* z = static_cast<const T*>(p.z) + (on ? n : 0) * p.stride;
  Stat a{-INFINITY, 0.0f, 0.0f};
  uint32_t best = static_cast<uint32_t>(lane);   // the first of the lane's chunks, where it has any
  for (int64_t c0 = 0; c0 * V < p.V; c0 += LPR * kAhead) {   // uniform, as is whether any lane has a chunk
    Vec<T, V> x[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t c = c0 + u * LPR + lane;
      if ((c0 + u * LPR) * V < p.V) x[u] = load_row<T, V>(z + c * V, p.V - c * V, from_f32<T>(-INFINITY));
    }
    float m = a.m;
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if ((c0 + u * LPR) * V < p.V) {
        float cm = -INFINITY;
#pragma unroll
        for (int e = 0; e < V; ++e) cm = fmaxf(cm, x[u].get(e));
        if (TOP) best = cm > m ? static_cast<uint32_t>(c0) + u * LPR + lane : best;
        m = fmaxf(m, cm);
      }
    if (m > a.m) rebase(a, m);
    const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if ((c0 + u * LPR) * V < p.V)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float t = x[u].get(e) - base, w = hw_exp2(kLog2e * t);
          a.z += w;
          a.s = weighted(w, t, a.s);
        }
  }
  const float own = a.m;
  join<LPR>(a, sh);
  const bool none = a.z == 0.0f;
  const float ls = kLn2 * hw_log2(a.z);
  if (lane == 0 && on) {
    if (p.lse) p.lse[n] = none ? -INFINITY : a.m + ls;
    if (p.entropy) p.entropy[n] = none ? 0.0f : ls - a.s / a.z;
    if (p.logp) {
      const int64_t t = target_of(p.targets, p.tbytes, n);
      p.logp[n] = t < 0 ? 0.0f : t >= p.V ? NAN : none ? -INFINITY : (to_f32(z[t]) - a.m) - ls;
    }
  }
  if constexpr (TOP) {
    __shared__ TopShared<LPR> top;
    top_of<T, LPR>(p, z, n, static_cast<int64_t>(lane) * V < p.V ? rank_key(own, best) : 0, a.m, ls, none, top);
  }
}

struct LogpGradArgs {
  const void* z;
  int64_t stride, N, V;
  const void* targets;
  int tbytes;
  const float *lse, *entropy, *g_logp, *g_entropy;
  void* dz;
  int64_t dstride, segments;
};

constexpr int kGradThreads = 256;

// f(j, chunk, columns from j on) for each of a lane's chunks of a row, kAhead loads at a time
template <typename T, int LPR, bool LAST, class F> DEV void each_chunk(const T* z, int64_t columns, int lane, F f) {
  constexpr int V = 16 / sizeof(T), S = LPR * V;
  int64_t j = static_cast<int64_t>(lane) * V, left = columns;   // left: from the round's first column
#pragma unroll 1
  for (; left >= kAhead * S; left -= kAhead * S, j += kAhead * S) {   // whole chunks: no lane tests for a row's end
    Vec<T, V> x[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) x[u] = load_row<T, V, LAST>(z + j + u * S, V, T{});
#pragma unroll
    for (int u = 0; u < kAhead; ++u) f(j + u * S, x[u], V);
  }
  Vec<T, V> x[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (j + u * S < columns) x[u] = load_row<T, V, LAST>(z + j + u * S, columns - j - u * S, from_f32<T>(-INFINITY));
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (j + u * S < columns) f(j + u * S, x[u], columns - j - u * S);
}

// ln sum_j e^{z_j - lse} of a row: what the rounding of its lse left out, 0 up to half a unit of lse (up to ln V where lse
// has no bits left for ln V).  More than a unit and 2^-18 (for the sums' own errors) is no rounding: the lse is that of
// other logits, of a row that these are a part of for instance, and is taken as given.  The same value for each of the row's
// LPR lanes, in a fixed order.
template <typename T, int LPR>
DEV float log_rest(const T* z, int64_t columns, float lse, int lane, float (&sh)[LPR > WAVE ? LPR / WAVE : 1]) {
  constexpr int V = 16 / sizeof(T);
  float s = 0.0f;
  each_chunk<T, LPR, false>(z, columns, lane, [&](int64_t, const Vec<T, V>& x, int64_t) {
#pragma unroll
    for (int e = 0; e < V; ++e) s += hw_exp2(kLog2e * (x.get(e) - lse));
  });
  s = LPR == 16 ? row_sum(s) : wave_sum(s);
  if constexpr (LPR > WAVE) {
    if (threadIdx.x % WAVE == 0) sh[threadIdx.x / WAVE] = s;
    __syncthreads();
    s = sh[0];
#pragma unroll
    for (int w = 1; w < LPR / WAVE; ++w) s += sh[w];
  }
  const float rest = kLn2 * hw_log2(s);
  return fabsf(rest) > fmaf(0x1p-23f, fabsf(lse), 0x1p-18f) ? 0.0f : rest;   // a NaN stays
}

// LPR lanes of one row write a segment of kAhead chunks each.  p_j = e^{z_j - lse}, where lse is one float32: half a unit of it
// is a relative error of every p_j, 16 u (u = 2^-24) for |lse| up to kLseExact, as much as the rounding of z - lse costs a
// token of p = e^-16.  Beyond that the error would grow with an offset that the logits have in common and that the softmax
// does not see, up to a row of the type's lowest values, whose lse has lost all of ln V.  The normaliser of such a row is
// summed again about lse, and one workgroup then writes the whole row (which may be the logits' own: nothing is written before
// all of it has been summed).  For all rows below and all above the bound: float32 4096 x 32000 174 and 235 us, bf16 4096 x 131072
// 342 and 492, 65536 x 256 14.2 and 18.7, 32 x 50001 4.4 and 13.6.
constexpr float kLseExact = 32.0f;
template <typename T, int LPR>
__global__ __launch_bounds__(kGradThreads) void k_logp_grad(const LogpGradArgs p) {
  constexpr int V = 16 / sizeof(T), RG = kGradThreads / LPR;
  __shared__ float sh[LPR > WAVE ? LPR / WAVE : 1];
  const int lane = threadIdx.x % LPR;
  const int64_t block = blockIdx.x, rows = block / p.segments, seg = block - rows * p.segments;
  const int64_t n = LPR == kGradThreads ? rows : rows * RG + threadIdx.x / LPR;   // scalar where a row has the workgroup
  if (n >= p.N) return;
  const T* z = static_cast<const T*>(p.z) + n * p.stride;
  T* dz = static_cast<T*>(p.dz) + n * p.dstride;
  const float lse = p.lse[n];
  const bool again = fabsf(lse) > kLseExact && fabsf(lse) < INFINITY;   // the same for all lanes of the row
  // the row's one workgroup, another segment's from row to row and from one run of rows to the next: each row's first would be
  // on one XCD where there are 8 or 16 segments (1258 us in place of 235), and with the row number alone on a few of its CUs (511)
  if (LPR == kGradThreads && again && seg != (rows + rows / p.segments) % p.segments) return;
  Vec<T, V> x[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    const int64_t j = ((seg * kAhead + u) * LPR + lane) * V;
    if (j < p.V) x[u] = load_row<T, V, true>(z + j, p.V - j, T{});
  }
  const int64_t t = p.targets ? target_of(p.targets, p.tbytes, n) : -1;
  const float g = t < 0 ? 0.0f : t >= p.V ? NAN : p.g_logp[n];
  const float ge = p.g_entropy ? p.g_entropy[n] : 0.0f, h = p.g_entropy ? p.entropy[n] : 0.0f;
  const bool none = lse == -INFINITY;
  const auto write = [&](int64_t j, const Vec<T, V>& v, int64_t left, float rest) {
    float o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float l = none ? -INFINITY : (v.get(e) - lse) - rest, q = hw_exp2(kLog2e * l);
      // below -104 q is 0, and ge l stays finite up to ge = 1e34
      o[e] = -q * fmaf(ge, fmaxf(l, -1e4f) + h, g);
    }
    const int64_t at = t - j;
    if (at >= 0 && at < V && !none)
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e == at) o[e] += g;
    store_row<T, V>(dz + j, left, o);
  };
  if (again) {
    const float rest = log_rest<T, LPR>(z, p.V, lse, lane, sh);
    each_chunk<T, LPR, true>(z, p.V, lane, [&](int64_t j, const Vec<T, V>& v, int64_t left) { write(j, v, left, rest); });
    return;
  }
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    const int64_t j = ((seg * kAhead + u) * LPR + lane) * V;
    if (j >= p.V) break;
    write(j, x[u], p.V - j, 0.0f);
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
  if (!grid_ok(N, V <= 4096 ? 64 : V <= 32768 ? 256 : 1024)) return PARARNN_ERR_UNSUPPORTED;   // the lanes of a row
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
  const LogpArgs a{logits, stride, N, V, targets, target_bytes, top, lse, logp, entropy, top_logp, top_ids};
  hipStream_t st = static_cast<hipStream_t>(stream);
  const auto run = [&](auto t, auto lanes, auto alt) {
    constexpr int LPR = decltype(lanes)::value, NT = LPR > WAVE ? LPR : WAVE;
    k_logp<decltype(t), LPR, decltype(alt)::value><<<static_cast<unsigned>(ceil_div(N, NT / LPR)), NT, 0, st>>>(a);
  };
  const auto sized = [&](auto t) {
    const auto alt = [&](auto lanes) {
      if (top) run(t, lanes, std::true_type{});
      else run(t, lanes, std::false_type{});
    };
    // Lanes of a row.  Few rows leave CUs idle, so theirs are read by more lanes: 32 rows, 20 alternatives, bf16: V = 3000
    // 8.2 us with 64 lanes and 6.7 with 256; V = 24000 9.9 with 256 and 8.8 with 1024 (float32 11.7 and 9.4).  Many rows fill
    // the chip either way and waste less of a row's end: 4096 rows: V = 3000 16.5 and 19.7; V = 24000 50 and 79.  512 rows of
    // 1024 lanes are what the chip holds at once: V = 24000 12.0 and 11.2 at 512, 14.1 and 16.0 at 640.  (At V = 3000 the lines
    // cross later: 8.8 and 8.2 at 1024, 10.1 and 11.8 at 2048.)
    const bool few = N <= 512;
    if (V <= 512 && !top) run(t, std::integral_constant<int, 16>{}, std::false_type{});
    else if (V <= (few ? 2048 : 4096)) alt(std::integral_constant<int, 64>{});
    else if (V <= (few ? 16384 : 32768)) alt(std::integral_constant<int, 256>{});
    else alt(std::integral_constant<int, 1024>{});
  };
  if (dtype == PARARNN_BF16) sized(bf16{});
  else sized(float{});
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
  hipStream_t st = static_cast<hipStream_t>(stream);
  const auto run = [&](auto t, auto lanes) {
    using T = decltype(t);
    constexpr int LPR = decltype(lanes)::value;
    constexpr int RG = kGradThreads / LPR;
    const int64_t segments = ceil_div(V, LPR * kAhead * 16 / static_cast<int64_t>(sizeof(T)));
    const int64_t most = INT64_C(0xffffffff) / kGradThreads / segments * RG;   // rows of a launch; V < 2^31: at least 32
    for (int64_t n = 0; n < N; n += most) {
      const int64_t rows = std::min(N - n, most);
      const LogpGradArgs a{static_cast<const T*>(logits) + n * stride, stride, rows, V,
                           targets ? static_cast<const char*>(targets) + n * target_bytes : nullptr, target_bytes, lse + n,
                           entropy ? entropy + n : nullptr, g_logp ? g_logp + n : nullptr, g_entropy ? g_entropy + n : nullptr,
                           static_cast<T*>(d_logits) + n * d_stride, d_stride, segments};
      k_logp_grad<T, LPR><<<static_cast<unsigned>(ceil_div(rows, RG) * segments), kGradThreads, 0, st>>>(a);
    }
    return launched();
  };
  const auto sized = [&](auto t) {
    const int64_t chunks = ceil_div(V, 16 / static_cast<int64_t>(sizeof(t)));
    if (chunks <= 16 * kAhead) return run(t, std::integral_constant<int, 16>{});
    if (chunks <= 64 * kAhead) return run(t, std::integral_constant<int, 64>{});
    return run(t, std::integral_constant<int, 256>{});
  };
  return dtype == PARARNN_BF16 ? sized(bf16{}) : sized(float{});
}
