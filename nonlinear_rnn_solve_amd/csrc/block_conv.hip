// block_conv.hip -- the short causal convolution of pararnn_block.h and its gradients.
//
//   p_t = bias + sum_k w[k] x_{t-K+1+k},  y_t = p_t sig(p_t);  K - 1 steps of state stand before each sequence

#include <type_traits>

#include "block_common.h"

namespace lm {

// A thread holds V channels and walks L consecutive steps with the K - 1 steps before them in registers, so every input is
// read once, but for the K - 1 rows that a chunk shares with the next (from the caches).  Threads are numbered over channels
// first, then chunks, then rows: narrow widths fill their waves with several chunks.  Bound by memory: B = 2, T = 4096, D = 4096,
// K = 4, bf16: 30 us forward (134 MB, 4.5 TB/s), 63 us backward (201 MB, 3.2 TB/s; of a fresh dx and three planes at once).
constexpr int V = 4, U = 4;     // channels of a thread; rows it has in flight

struct ConvArgs {
  const void* x;
  int64_t sx[2];
  const float *weight, *bias, *state;
  Seqs seqs;
  int64_t B, T, D;
  int64_t quads, chunks, main, threads;   // threads of a row and chunk, chunks of a row, threads that walk, all threads
  int32_t L, silu;
  void* y;
  int64_t sy[2];
  float* last;
  bool last_here;               // one chunk a row and no offsets: the walk ends with the state that leaves
};

struct ConvGradArgs {
  ConvArgs f;
  const void* dy;
  const float* d_last;
  void* dx;
  int64_t sdy[2], sdx[2];
  float* part;                  // [B groups][K + 1][D]: sums over a group of chunks, the bias's last; or null
  float* d_state;
  int32_t log_quads;            // a workgroup's threads are 2^log_quads quads by chunks
  int64_t groups, qgroups;      // groups of chunks of a row, of quads
};

// V float32 values of a row of n channels, `fill`ed past its end
DEV void load_f(const float* p, int64_t n, float (&v)[V]) {
  const Vec<float, V> r = load_row<float, V>(p, n, 0.0f);
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = r.get(i);
}
DEV void store_f(float* p, int64_t n, const float (&v)[V]) { store_row<float, V>(p, n, v); }

// what a thread's channels and place are
struct Place {
  int64_t b, chunk, d, left;    // left: channels from d on
};
DEV Place place(int64_t id, int64_t quads, int64_t middle, int64_t D) {
  const int64_t q = id % quads, r = id / quads;
  return {r / middle, r % middle, q * V, D - q * V};
}

// weights as w[k][channel]
template <int K> DEV void load_taps(const ConvArgs& p, int64_t d, int64_t left, float (&w)[K][V], float (&bias)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    bias[i] = p.bias && i < left ? p.bias[d + i] : 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) w[k][i] = i < left ? p.weight[(d + i) * K + k] : 0.0f;
  }
}

// row r of the K - 1 before step t of sequence j, which begins at s <= t: of x, or of the state
template <typename T, int K>
DEV void history(const ConvArgs& p, int64_t b, int64_t j, int64_t s, int64_t t, int64_t d, int64_t left, float (&win)[K][V]) {
#pragma unroll
  for (int i = 0; i + 1 < K; ++i) {
    const int64_t row = t - (K - 1) + i;
    if (row >= s) {
      const Vec<T, V> v = load_row<T, V>(static_cast<const T*>(p.x) + b * p.sx[0] + row * p.sx[1] + d, left, T{});
#pragma unroll
      for (int c = 0; c < V; ++c) win[i][c] = v.get(c);
    } else if (p.state) {
      load_f(p.state + ((b * p.seqs.n + j) * (K - 1) + (row - s + K - 1)) * p.D + d, left, win[i]);
    } else {
#pragma unroll
      for (int c = 0; c < V; ++c) win[i][c] = 0.0f;
    }
  }
}

// the state that leaves sequence j: the last K - 1 steps of its state and its own steps together; all is read before anything
// is written, since `last` may be the state itself
template <typename T, int K> DEV void leave(const ConvArgs& p, int64_t b, int64_t j, int64_t d, int64_t left) {
  if constexpr (K > 1) {
    const int64_t s = p.seqs.begin(j), e = p.seqs.end(j);
    float win[K][V];
    history<T, K>(p, b, j, s, e < s ? s : e, d, left, win);
#pragma unroll
    for (int i = 0; i + 1 < K; ++i) store_f(p.last + ((b * p.seqs.n + j) * (K - 1) + i) * p.D + d, left, win[i]);
  }
}

template <typename T, int K, bool SEG>
__global__ __launch_bounds__(256) void k_conv(const ConvArgs p) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (id >= p.threads) return;
  if (id >= p.main) {
    const Place q = place(id - p.main, p.quads, p.seqs.n, p.D);
    leave<T, K>(p, q.b, q.chunk, q.d, q.left);
    return;
  }
  const Place q = place(id, p.quads, p.chunks, p.D);
  const int64_t t0 = q.chunk * p.L;
  const int steps = static_cast<int>(p.T - t0 < p.L ? p.T - t0 : p.L);
  float w[K][V], bias[V], win[K][V];
  load_taps<K>(p, q.d, q.left, w, bias);
  int64_t j = 0, s = 0;
  int next = INT_MAX;           // steps from t0 on to the first of the next sequence
  const auto find = [&](int64_t t) {
    j = p.seqs.of(t);
    s = p.seqs.begin(j);
    s = s < t ? s : t;
    const int64_t e = p.seqs.end(j) - t0;
    next = e < steps ? static_cast<int>(e) : INT_MAX;
  };
  if constexpr (SEG) find(t0);
  history<T, K>(p, q.b, j, s, t0, q.d, q.left, win);
  const T* x = static_cast<const T*>(p.x) + q.b * p.sx[0] + t0 * p.sx[1] + q.d;
  T* y = static_cast<T*>(p.y) + q.b * p.sy[0] + t0 * p.sy[1] + q.d;
  for (int i0 = 0; i0 < steps; i0 += U) {
    Vec<T, V> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u < steps) v[u] = load_row<T, V>(x + (i0 + u) * p.sx[1], q.left, T{});
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u >= steps) break;
      if constexpr (SEG) {
        if (i0 + u == next) {
          find(t0 + i0 + u);
          history<T, K>(p, q.b, j, s, t0 + i0 + u, q.d, q.left, win);
        }
      }
      float o[V];
#pragma unroll
      for (int c = 0; c < V; ++c) {
        win[K - 1][c] = v[u].get(c);
        float a = bias[c];
#pragma unroll
        for (int k = 0; k < K; ++k) a = fmaf(w[k][c], win[k][c], a);
        o[c] = p.silu ? silu(a) : a;
#pragma unroll
        for (int k = 0; k + 1 < K; ++k) win[k][c] = win[k + 1][c];
      }
      store_row<T, V>(y + (i0 + u) * p.sy[1], q.left, o);
    }
  }
  if (!SEG && p.last_here) {
#pragma unroll
    for (int i = 0; i + 1 < K; ++i) store_f(p.last + (q.b * (K - 1) + i) * p.D + q.d, q.left, win[i]);
  }
}

// Gradients.  dp_t = dy_t silu'(p_t);  a row's gradient is sum_k w[k] dp of the step k taps later, within its sequence, plus
// d_last where it leaves as state.  A thread walks each sequence's part of its chunk [a, e) and the K - 1 steps after it, whose
// dp it needs too (computed twice, by this chunk and the next), and gives out the gradient of the step K - 1 before; at a
// sequence's start those are its state's.  A workgroup's threads are some quads of channels by as many chunks as make 256: it
// adds up the parameters' sums of its chunks.
template <typename T, int K, bool SEG>
__global__ __launch_bounds__(256) void k_conv_vjp(const ConvGradArgs g) {
  const ConvArgs& p = g.f;
  if (blockIdx.x >= p.main) {   // the states of empty sequences
    const int64_t id = (blockIdx.x - p.main) * 256 + threadIdx.x;
    if (id >= p.B * p.seqs.n * p.quads) return;
    const Place q = place(id, p.quads, p.seqs.n, p.D);
    if (p.seqs.end(q.chunk) > p.seqs.begin(q.chunk)) return;
    for (int i = 0; i + 1 < K; ++i) {
      const int64_t at = ((q.b * p.seqs.n + q.chunk) * (K - 1) + i) * p.D + q.d;
      float v[V] = {};
      if (g.d_last) load_f(g.d_last + at, q.left, v);
      store_f(g.d_state + at, q.left, v);
    }
    return;
  }
  const int lane_q = threadIdx.x & ((1 << g.log_quads) - 1), lane_c = threadIdx.x >> g.log_quads, rows = 256 >> g.log_quads;
  const int64_t qg = blockIdx.x % g.qgroups, rest = blockIdx.x / g.qgroups, b = rest / g.groups, group = rest - b * g.groups;
  Place q{b, group * rows + lane_c, ((qg << g.log_quads) + lane_q) * V, 0};
  const bool there = q.d < p.D && q.chunk < p.chunks;
  q.left = p.D - q.d;
  const int64_t t0 = q.chunk * p.L, t1 = !there ? t0 : p.T - t0 < p.L ? p.T : t0 + p.L;
  float w[K][V], bias[V], dw[K][V] = {}, db[V] = {};
  load_taps<K>(p, q.d, there ? q.left : 0, w, bias);
  const T* x = static_cast<const T*>(p.x) + q.b * p.sx[0] + q.d;
  const T* dy = static_cast<const T*>(g.dy) + q.b * g.sdy[0] + q.d;
  T* dx = static_cast<T*>(g.dx) + q.b * g.sdx[0] + q.d;
  for (int64_t a = t0; a < t1;) {
    int64_t j = 0, s = 0, end = p.T;
    if constexpr (SEG) {
      j = p.seqs.of(a);
      s = p.seqs.begin(j);
      s = s < a ? s : a;
      end = p.seqs.end(j);
      end = end > a ? end : a + 1;
    }
    const int64_t e = end < t1 ? end : t1;
    float win[K][V], ring[K][V] = {};
    history<T, K>(p, q.b, j, s, a, q.d, q.left, win);
    const int count = static_cast<int>(e - a) + K - 1;                          // steps of the walk
    const int have = static_cast<int>(end - a < count ? end - a : count);       // those inside the sequence
    for (int i0 = 0; i0 < count; i0 += U) {
      Vec<T, V> vx[U], vd[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u < have) {
          vx[u] = load_row<T, V>(x + (a + i0 + u) * p.sx[1], q.left, T{});
          vd[u] = load_row<T, V>(dy + (a + i0 + u) * g.sdy[1], q.left, T{});
        }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u;
        if (i >= count) break;
        float out[V];
        const bool in = i < have, mine = i < static_cast<int>(e - a);
#pragma unroll
        for (int c = 0; c < V; ++c) {
          float dp = 0.0f;
          if (in) {
            win[K - 1][c] = vx[u].get(c);
            dp = vd[u].get(c);
            if (p.silu) {
              float z = bias[c];
#pragma unroll
              for (int k = 0; k < K; ++k) z = fmaf(w[k][c], win[k][c], z);
              dp *= silu_slope(z, sigmoid(z));
            }
            if (mine) {
              db[c] += dp;
#pragma unroll
              for (int k = 0; k < K; ++k) dw[k][c] = fmaf(dp, win[k][c], dw[k][c]);
            }
#pragma unroll
            for (int k = 0; k + 1 < K; ++k) win[k][c] = win[k + 1][c];
          }
#pragma unroll
          for (int k = 0; k + 1 < K; ++k) ring[k][c] = ring[k + 1][c];
          ring[K - 1][c] = dp;
          out[c] = 0.0f;
#pragma unroll
          for (int k = 0; k < K; ++k) out[c] = fmaf(w[k][c], ring[K - 1 - k][c], out[c]);
        }
        const int64_t t = a + i - (K - 1);                  // the step that this gradient belongs to
        const bool state = t < a;
        if (state && (a != s || !g.d_state)) continue;
        if (g.d_last && t >= end - (K - 1)) {
          float v[V];
          load_f(g.d_last + ((q.b * p.seqs.n + j) * (K - 1) + (t - end + K - 1)) * p.D + q.d, q.left, v);
#pragma unroll
          for (int c = 0; c < V; ++c) out[c] += v[c];
        }
        if (state) store_f(g.d_state + ((q.b * p.seqs.n + j) * (K - 1) + (t - s + K - 1)) * p.D + q.d, q.left, out);
        else store_row<T, V>(dx + t * g.sdx[1], q.left, out);
      }
    }
    a = e;
  }
  if (g.part) {                 // uniform
    __shared__ float4 sums[256];
    float* part = g.part + (b * g.groups + group) * (K + 1) * p.D + q.d;
#pragma unroll
    for (int k = 0; k <= K; ++k) {
      const float* v = k < K ? dw[k < K ? k : 0] : db;
      sums[threadIdx.x] = make_float4(v[0], v[1], v[2], v[3]);
      __syncthreads();
      if (lane_c == 0 && q.d < p.D) {
        float o[V] = {};
        for (int c = 0; c < rows; ++c) {
          const float4 e = sums[(c << g.log_quads) + lane_q];
          o[0] += e.x, o[1] += e.y, o[2] += e.z, o[3] += e.w;
        }
        store_f(part + k * p.D, q.left, o);
      }
      __syncthreads();
    }
  }
}

// where the column sums [K + 1][D] go: d_weight [D][K] and d_bias [D]
struct ToTaps {
  int64_t D;
  int32_t K;
  float *d_weight, *d_bias;
  DEV void operator()(int64_t, int64_t i, float v) const {
    const int64_t k = i / D, d = i - k * D;
    float* to = k < K ? d_weight : d_bias;
    if (to) to[k < K ? d * K + k : d] = v;
  }
};

// ---------------- host ----------------
// Steps of a chunk: as many as leave `want` threads, since longer chunks read and compute fewer shared rows.  Forward with 2^16, 2^18
// and 2^20 threads: 35.7, 21.5, 21.6 us (T = 81708, D = 145, K = 5, bf16), 25.2, 28.1, 28.1 (B = 8, T = 2048, D = 1000, K = 4, f32).
// Gradient with 2^15, 2^17 and 2^19: 110, 112, 124 and 96, 75, 90 there, 81, 79, 86 at B = 2, T = 4096, D = 4096, K = 4, bf16.
inline int32_t chunk_steps(int64_t B, int64_t T, int64_t D, int64_t want, int32_t most) {
  const int64_t quads = ceil_div(D, V);
  int32_t L = most;
  while (L > 8 && B * quads * ceil_div(T, L) < want) L /= 2;
  return L;
}
constexpr int64_t kThreads = 1 << 18, kGradThreads = 1 << 17;
inline int32_t forward_steps(int64_t B, int64_t T, int64_t D) { return chunk_steps(B, T, D, kThreads, 32); }
inline int32_t gradient_steps(int64_t B, int64_t T, int64_t D) { return chunk_steps(B, T, D, kGradThreads, 64); }

static bool sizes_ok(int64_t B, int64_t T, int64_t D, int64_t K) {
  // every product of sizes fits, also where a third one is zero
  return K >= 1 && sizes_fit(B, T, D) && sizes_fit(B, T) && sizes_fit(T, D) && sizes_fit(B, D, 8) && sizes_fit(D, 9);
}
static bool problem_ok(const pararnn_block_conv* q) {
  if (!q || !dtype_ok(q->dtype) || (q->silu != 0 && q->silu != 1) || !sizes_ok(q->B, q->T, q->D, q->K)) return false;
  const size_t e = dtype_size(q->dtype);
  const bool any = q->B > 0 && q->D > 0, steps = any && q->T > 0;
  if (!ptr_ok(q->x, e, steps) || !ptr_ok(q->weight, 4, any) || !ptr_ok(q->bias, 4, false) || !ptr_ok(q->state, 4, false) ||
      !ptr_ok(q->cu_seqlens, 4, false))
    return false;
  if (q->cu_seqlens && (q->n_seqs < 1 || q->T > INT32_MAX)) return false;
  if (q->cu_seqlens && !sizes_fit(q->n_seqs, q->D, 8)) return false;
  if (q->cu_seqlens && q->B && q->n_seqs * q->D * 8 > INT64_MAX / 16 / q->B) return false;
  return plane_ok(q->B, q->sx[0]) && plane_ok(q->T, q->sx[1]);
}
static ConvArgs conv_args(const pararnn_block_conv* q) {
  ConvArgs p{};
  p.x = q->x;
  p.sx[0] = q->sx[0], p.sx[1] = q->sx[1];
  p.weight = q->weight, p.bias = q->bias, p.state = q->state;
  p.seqs = {q->cu_seqlens, q->cu_seqlens ? q->n_seqs : 1, q->T};
  p.B = q->B, p.T = q->T, p.D = q->D;
  p.quads = ceil_div(q->D, V);
  p.silu = q->silu;
  return p;
}

template <typename T, int K> static pararnn_status forward_k(const ConvArgs& p, hipStream_t stream) {
  const int64_t blocks = ceil_div(p.threads, 256);
  if (p.seqs.cu) k_conv<T, K, true><<<dim3(static_cast<uint32_t>(blocks)), dim3(256), 0, stream>>>(p);
  else k_conv<T, K, false><<<dim3(static_cast<uint32_t>(blocks)), dim3(256), 0, stream>>>(p);
  return launched();
}
template <typename T, int K> static pararnn_status backward_k(const ConvGradArgs& g, hipStream_t stream) {
  const int64_t blocks = g.f.threads;
  if (g.f.seqs.cu) k_conv_vjp<T, K, true><<<dim3(static_cast<uint32_t>(blocks)), dim3(256), 0, stream>>>(g);
  else k_conv_vjp<T, K, false><<<dim3(static_cast<uint32_t>(blocks)), dim3(256), 0, stream>>>(g);
  return launched();
}
template <int K, typename A> static pararnn_status by_type(int dtype, const A& a, hipStream_t stream) {
  if constexpr (std::is_same_v<A, ConvArgs>)
    return dtype == PARARNN_BF16 ? forward_k<bf16, K>(a, stream) : forward_k<float, K>(a, stream);
  else
    return dtype == PARARNN_BF16 ? backward_k<bf16, K>(a, stream) : backward_k<float, K>(a, stream);
}
template <typename A> static pararnn_status dispatch(int64_t K, int dtype, const A& a, hipStream_t stream) {
  switch (K) {
    case 1: return by_type<1>(dtype, a, stream);
    case 2: return by_type<2>(dtype, a, stream);
    case 3: return by_type<3>(dtype, a, stream);
    case 4: return by_type<4>(dtype, a, stream);
    case 5: return by_type<5>(dtype, a, stream);
    case 6: return by_type<6>(dtype, a, stream);
    case 7: return by_type<7>(dtype, a, stream);
    default: return by_type<8>(dtype, a, stream);
  }
}

// the gradient's workgroups, and the floats of its workspace: groups' sums and the column sums' scratch
struct Parts {
  int32_t L, log_quads;
  int64_t chunks, groups, qgroups, rows, cols, part, scratch;
};
static Parts parts(int64_t B, int64_t T, int64_t D, int64_t K) {
  Parts s;
  s.L = gradient_steps(B, T, D);
  s.chunks = ceil_div(T, s.L);
  s.log_quads = 0;
  while (s.log_quads < 5 && (INT64_C(1) << s.log_quads) < ceil_div(D, V)) ++s.log_quads;
  s.groups = ceil_div(s.chunks, 256 >> s.log_quads);
  s.qgroups = ceil_div(ceil_div(D, V), INT64_C(1) << s.log_quads);
  s.rows = B * s.groups;
  s.cols = D * (K + 1);
  s.part = ceil_div(s.rows * s.cols, 64) * 64;
  s.scratch = colsum_floats(s.rows, s.cols);
  return s;
}

}  // namespace lm

using namespace lm;

extern "C" size_t pararnn_block_conv_workspace_bytes(int64_t B, int64_t T, int64_t D, int64_t K) {
  if (!sizes_ok(B, T, D, K) || K > PARARNN_BLOCK_MAX_TAPS) return 0;
  const Parts s = parts(B, T, D, K);
  return static_cast<size_t>(s.part + s.scratch) * sizeof(float);
}

extern "C" pararnn_status pararnn_block_causal_conv(const pararnn_block_conv* q, void* y, const int64_t sy[2], float* last,
                                                    void* stream) {
  if (!problem_ok(q) || !sy || !plane_ok(q->B, sy[0]) || !plane_ok(q->T, sy[1])) return PARARNN_ERR_INVALID_ARG;
  const bool any = q->B > 0 && q->D > 0;
  if (!ptr_ok(y, dtype_size(q->dtype), any && q->T > 0) || !ptr_ok(last, 4, false)) return PARARNN_ERR_INVALID_ARG;
  if (q->K > PARARNN_BLOCK_MAX_TAPS) return PARARNN_ERR_UNSUPPORTED;
  if (!any) return PARARNN_OK;
  ConvArgs p = conv_args(q);
  p.y = y;
  p.sy[0] = sy[0], p.sy[1] = sy[1];
  p.last = q->K > 1 ? last : nullptr;
  p.L = forward_steps(p.B, p.T, p.D);
  p.chunks = ceil_div(p.T, p.L);
  p.last_here = p.last && !p.seqs.cu && p.chunks == 1;
  p.main = p.B * p.chunks * p.quads;
  // the states that leave: by the walk itself, by more threads of the launch, or, where they take the place of the states that
  // the walk reads, by a launch of their own
  const int64_t leaving = p.last && !p.last_here ? p.B * p.seqs.n * p.quads : 0;
  const bool apart = leaving && p.last == p.state && p.main > 0;
  p.threads = p.main + (apart ? 0 : leaving);
  if (!grid_ok(ceil_div(p.threads, 256), 256) || !grid_ok(ceil_div(leaving, 256), 256)) return PARARNN_ERR_UNSUPPORTED;
  if (p.threads == 0) return PARARNN_OK;
  const auto s = static_cast<hipStream_t>(stream);
  pararnn_status r = dispatch(q->K, q->dtype, p, s);
  if (r == PARARNN_OK && apart) {
    p.main = 0;
    p.threads = leaving;
    r = dispatch(q->K, q->dtype, p, s);
  }
  return r;
}

extern "C" pararnn_status pararnn_block_causal_conv_vjp(const pararnn_block_conv* q, const pararnn_block_conv_grad* grad, void* ws,
                                                        size_t ws_bytes, void* stream) {
  if (!problem_ok(q) || !grad) return PARARNN_ERR_INVALID_ARG;
  const size_t e = dtype_size(q->dtype);
  const bool any = q->B > 0 && q->D > 0, steps = any && q->T > 0;
  if (!ptr_ok(grad->dy, e, steps) || !ptr_ok(grad->d_x, e, steps) || !ptr_ok(grad->d_last, 4, false) ||
      !ptr_ok(grad->d_weight, 4, false) || !ptr_ok(grad->d_bias, 4, false) || !ptr_ok(grad->d_state, 4, false))
    return PARARNN_ERR_INVALID_ARG;
  if (!plane_ok(q->B, grad->sdy[0]) || !plane_ok(q->T, grad->sdy[1]) || !plane_ok(q->B, grad->sdx[0]) ||
      !plane_ok(q->T, grad->sdx[1]))
    return PARARNN_ERR_INVALID_ARG;
  if (q->K > PARARNN_BLOCK_MAX_TAPS) return PARARNN_ERR_UNSUPPORTED;
  const bool params = grad->d_weight || grad->d_bias;
  if (params && q->D > 0 && !ws_ok(ws, ws_bytes, pararnn_block_conv_workspace_bytes(q->B, q->T, q->D, q->K)))
    return PARARNN_ERR_WORKSPACE;
  if (q->D == 0) return PARARNN_OK;
  ConvGradArgs g{};
  g.f = conv_args(q);
  ConvArgs& p = g.f;
  const Parts s = parts(p.B, p.T, p.D, q->K);
  p.L = s.L, p.chunks = s.chunks;
  g.log_quads = s.log_quads, g.groups = s.groups, g.qgroups = s.qgroups;
  p.main = s.rows * s.qgroups;  // workgroups here, and p.threads all of them
  g.dy = grad->dy, g.d_last = grad->d_last, g.dx = grad->d_x;
  for (int k = 0; k < 2; ++k) g.sdy[k] = grad->sdy[k], g.sdx[k] = grad->sdx[k];
  g.d_state = q->K > 1 ? grad->d_state : nullptr;
  float* base = static_cast<float*>(ws);
  if (params) g.part = base;
  p.threads = p.main + (g.d_state && (p.seqs.cu || p.T == 0) ? ceil_div(p.B * p.seqs.n * p.quads, 256) : 0);
  if (!grid_ok(p.threads, 256)) return PARARNN_ERR_UNSUPPORTED;
  const auto st = static_cast<hipStream_t>(stream);
  if (p.threads) {
    const pararnn_status r = dispatch(q->K, q->dtype, g, st);
    if (r != PARARNN_OK) return r;
  }
  if (!params) return PARARNN_OK;
  if (!colsum(base, s.rows, s.cols, ToTaps{q->D, static_cast<int32_t>(q->K), grad->d_weight, grad->d_bias}, base + s.part, st))
    return PARARNN_ERR_UNSUPPORTED;
  return launched();
}

extern "C" int pararnn_block_abi_version(void) { return PARARNN_BLOCK_ABI_VERSION; }
