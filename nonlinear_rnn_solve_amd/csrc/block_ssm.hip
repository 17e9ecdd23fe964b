// block_ssm.hip -- the selective state space scan of pararnn_block.h and its gradients.
//
//   dt = softplus(delta + dt_bias),  h_t[n] = exp(dt A[n]) h_{t-1}[n] + dt x_t B_t[n],
//   y_t = (sum_n C_t[n] h_t[n] + skip x_t) silu(z_t)

#include <type_traits>

#include "block_common.h"

namespace lm {

// ------------------------------------------------------------------------------------------------
// A workgroup holds 64 channels of one row, a lane a channel; its WV waves split the states, NS each.  So B_t and C_t are the
// same for all lanes of a wave and x, delta and z the same for all its states: per step and state a lane takes one
// exponential and four other instructions, and what a channel's step takes once (softplus, SiLU) is shared out over the
// waves.  Time goes in tiles of CT steps: all waves load the tile's x, delta, z, B, C (those of the next tile are in flight
// while this one is walked), put dt, dt x, B and C in shared memory, walk the steps, leave their part of y there, and share out
// the sums.  B and C are then held one value a lane, replicated over the wave's four rows of 16 lanes, and reach the
// products by the row broadcast of their operand (no instruction, no access of its own).
//
// Bound by vector instructions: one exponential and four multiplications alone take 8.3 ns of a SIMD a wave's step and state (3.7 of
// them the exponential), the walk 20.  The rest is a step's reads and writes of shared memory, softplus, SiLU, conversions, and scalar
// registers kept in vector lanes (62 of them at N = 16, 73 in the gradient).  B = 2, T = 4096, D = 4096, N = 16, bf16 with z: 114 us for
// the segments' ends and 168 for the walk (268 MB; the planes alone 53 at a large copy's rate); the gradient 108 and 550 (470 MB, 92).
//
// Few rows and channels leave the chip empty, so long rows are cut into segments of whole tiles.  One launch finds what each
// segment leaves from a zero state and the sum of its dt (the decay over the segment is exp(A sum)), the next walks the
// segments, each from the state that the ones before it make together.  That walks everything but y twice, and pays where
// the workgroups without it are fewer than the chip holds.
// ------------------------------------------------------------------------------------------------
constexpr int CT = PARARNN_BLOCK_SSM_CHUNK;
constexpr int CH = 64;          // channels of a workgroup

struct SsmArgs {
  const void *x, *delta, *z, *b, *c;
  int64_t sx[2], sdelta[2], sz[2], sb[3], sc[3];
  const float *A, *skip, *dt_bias, *h0;
  Seqs seqs;
  int64_t B, D;
  int32_t T, N, G, tiles;       // tiles: of CT steps, of a row
  int32_t ctiles, group;        // channel tiles of a group, channels of a group
  int32_t S, per;               // segments of a row, tiles of a segment
  bool in_place;                // h_last takes h0's place
  void* y;
  int64_t sy[2];
  float *h_last, *carry;
  float *end, *sum, *head;      // [S][B][N][D], [S][B][D] of the segments; head: the last sequence's h0, in place only
};

struct SsmGradArgs {
  SsmArgs f;
  const float* carry;
  const void* dy;
  const float* d_last;
  void *dx, *ddelta, *dz;
  int64_t sdy[2], sdx[2], sddelta[2], sdz[2];
  float *d_h0;
  float *part_bc;               // [G ctiles][B][T][2][N]: a channel tile's sums for d_b and d_c
  float *part_A;                // [S B][N + 2][D]: for d_A, then d_skip and d_dt_bias
};

// the workgroup's channels, row and segment
struct Where {
  int32_t ct, g, d, left;       // channel tile over all groups, group, first channel, channels from it on in the group
  int64_t b;
  int32_t s;
};
DEV Where where(const SsmArgs& p) {
  const uint32_t n = static_cast<uint32_t>(p.ctiles * p.G), rows = blockIdx.x / n;
  Where w;
  w.ct = static_cast<int32_t>(blockIdx.x - rows * n);
  w.g = w.ct / p.ctiles;
  const int32_t in = (w.ct - w.g * p.ctiles) * CH;
  w.d = w.g * p.group + in;
  w.left = p.group - in;
  w.s = static_cast<int32_t>(rows / static_cast<uint32_t>(p.B));
  w.b = rows - w.s * p.B;
  return w;
}

// A launch's arguments, read anew: held in scalar registers over a tile they would not fit, and went through vector lanes (half of
// the instructions outside the walks).
template <typename A> DEV const A __attribute__((address_space(4)))* arguments() {
  auto p = (const A __attribute__((address_space(4)))*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return p;
}

// One channel's column of a plane, as its lane walks it tile by tile: the element of the tile's first step (made a vector
// register's, for the same reason) and the step's stride, which each tile sets.  Rows past the last step are read as the last, lanes
// past the last channel as the last: nothing branches, and what they give is left out later.  A tile's steps are less than 2^28
// elements apart (checked), so that 32 bits hold their offsets.
template <typename T> using Bits = std::conditional_t<sizeof(T) == 2, uint16_t, float>;
template <typename T> using Global = __attribute__((address_space(1))) Bits<T>;
template <typename T> DEV Global<T>* in_vector(const void* plane, int64_t at) {
  auto p = (Global<T>*)plane + at;
  asm("" : "+v"(p));
  return p;
}
DEV float value(float x) { return x; }
DEV float value(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }
template <typename T> struct Column {
  Global<T>* at;
  int32_t s;
  DEV Column(const void* plane, const int64_t (&st)[2], int64_t b, int64_t t, const Where& w, int lane)
      : at(in_vector<T>(plane, b * st[0] + t * st[1] + w.d + (lane < w.left ? lane : w.left - 1))), s(static_cast<int32_t>(st[1])) {}
  DEV void move(int32_t steps) { at += steps * s; }
  template <int E> DEV void load(int wave, int wv, int32_t steps, Bits<T> (&v)[E]) const {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int32_t t = wave + i * wv;
      v[i] = at[(t < steps ? t : steps - 1) * s];
    }
  }
  DEV void store(int32_t t, float x) const {
    if constexpr (sizeof(T) == 2) at[t * s] = bf16_bits(x);
    else at[t * s] = x;
  }
};

// lane k of each row of 16, for all lanes of the row
template <int K> DEV float row_lane(float v) { return dpp<0x150 + K>(v); }
// STEP's value n of NS, of registers that hold 16 / NS steps each
template <int NS, int STEP, int n> DEV float of_step(const float (&r)[NS]) {
  constexpr int SPR = 16 / NS;
  return row_lane<(STEP % SPR) * NS + n>(r[STEP / SPR]);
}
template <int I> using Int = std::integral_constant<int, I>;
template <int FROM, int TO, typename F> DEV void for_up(F&& f) {
  if constexpr (FROM < TO) {
    f(Int<FROM>{});
    for_up<FROM + 1, TO>(f);
  }
}

// What the threads of a workgroup load of a tile: wave w the steps w, w + WV, ... of its lanes' channels, and all together B and C.
template <typename T, int NS, int WV> struct Tile {
  static constexpr int E = CT / WV;                            // steps of a wave
  static constexpr int NP = NS * WV, TH = WV * WAVE;
  static constexpr int BC = (CT * NP + TH - 1) / TH;           // values of B and of C of a thread
};
// Some of a tile's B or C: thread k takes the values k, k + 64 WV, ... of [CT][NP]; zeros past the last step or state
template <typename T, int NS, int WV> struct Shared {
  using L = Tile<T, NS, WV>;
  Global<T>* at;                // of the tile's first value
  int32_t s, N;
  DEV Shared(const void* plane, const int64_t (&st)[3], int64_t b, int64_t t, int32_t g, int32_t n)
      : at(in_vector<T>(plane, b * st[0] + t * st[1] + g * st[2])), s(static_cast<int32_t>(st[1])), N(n) {}
  DEV void move(int32_t steps) { at += steps * s; }
  DEV void load(int32_t steps, Bits<T> (&v)[L::BC]) const {
#pragma unroll
    for (int i = 0; i < L::BC; ++i) {
      const int k = threadIdx.x + i * L::TH, t = k / L::NP, n = k - t * L::NP;
      v[i] = 0;
      if (t < steps && n < N) v[i] = at[t * s + n];
    }
  }
  static DEV void put(float* to, const Bits<T> (&v)[L::BC]) {
#pragma unroll
    for (int i = 0; i < L::BC; ++i) {
      const int k = threadIdx.x + i * L::TH;
      if (k < CT * L::NP) to[k] = value(v[i]);
    }
  }
};
// a wave's B or C of a tile, from [CT][NP] in shared memory: register r holds the steps r 16/NS and on
template <int NS, int NP> DEV void get_shared(const float* from, int wave, int lane, float (&r)[NS]) {
  constexpr int SPR = 16 / NS;
#pragma unroll
  for (int k = 0; k < NS; ++k) r[k] = from[(k * SPR + (lane & 15) / NS) * NP + wave * NS + (lane & 15) % NS];
}

// a wave's values of one step, the same for all lanes
template <int NS, int NP> DEV void step_values(const float* from, int wave, int t, float (&v)[NS]) {
  const float* q = from + t * NP + wave * NS;
  if constexpr (NS == 4) {
    const float4 r = *reinterpret_cast<const float4*>(q);
    v[0] = r.x, v[1] = r.y, v[2] = r.z, v[3] = r.w;
  } else if constexpr (NS == 2) {
    const float2 r = *reinterpret_cast<const float2*>(q);
    v[0] = r.x, v[1] = r.y;
  } else {
    v[0] = *q;
  }
}

// a wave's states of one channel, [n][D] (segments, carry) or [d][N] (h0, h_last); zeros past the last state
template <int NS> DEV void load_nd(const float* p, int32_t D, int32_t N, int n0, float (&v)[NS]) {
#pragma unroll
  for (int n = 0; n < NS; ++n) {
    const int32_t k = n0 + n < N ? n0 + n : N - 1;
    v[n] = p[k * D];
    v[n] = n0 + n < N ? v[n] : 0.0f;
  }
}
template <int NS> DEV void store_nd(float* p, int32_t D, int32_t N, int n0, bool in, const float (&v)[NS]) {
  if (!in) return;
#pragma unroll
  for (int n = 0; n < NS; ++n)
    if (n0 + n < N) p[(n0 + n) * D] = v[n];
}
template <int NS> DEV void load_dn(const float* p, int32_t N, int n0, float (&v)[NS]) {
  Vec<float, NS> r{};
  if (p) r = load_row<float, NS>(p + n0, N - n0, 0.0f);
#pragma unroll
  for (int n = 0; n < NS; ++n) v[n] = r.get(n);
}
template <int NS> DEV void store_dn(float* p, int32_t N, int n0, bool in, const float (&v)[NS]) {
  if (in) store_row<float, NS>(p + n0, N - n0, v);
}

// Where sequences begin in a tile, by step: which one does, and which one was before it (before[0]: the one of the step before the
// tile).  Every wave writes the same.
struct Marks {
  int32_t start[CT], before[CT + 1];
};
// The steps of a tile of `steps` at which a sequence begins, as bits, and whether one ends with the tile (bit 16); uniform.
DEV uint32_t marks_of(const Seqs& q, int32_t t0, int32_t steps, Marks& m) {
  const int32_t end = t0 + steps;
  if (!q.cu) return (t0 == 0 ? 1u : 0u) | (end == q.T ? 1u << CT : 0u);
  uint32_t bits = 0;
  int32_t now = t0 == 0 ? -1 : static_cast<int32_t>(q.of(t0 - 1)), t = 0, j = now + 1;
  for (; j < q.n; ++j) {
    t = j ? q.cu[j] : 0;
    if (t >= end) break;
    if (t >= t0) {
      if (!(bits >> (t - t0) & 1)) m.before[t - t0] = now;
      bits |= 1u << (t - t0);
      m.start[t - t0] = j;
    }
    now = j;
  }
  m.before[steps] = now;
  if (end == q.T || (j < q.n && t == end)) bits |= 1u << CT;
  return __builtin_amdgcn_readfirstlane(bits);
}
constexpr uint32_t kSteps = (1u << CT) - 1;
DEV int32_t uniform(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }

// Whether step t begins a sequence (t < T), or nothing follows (t = T)
DEV bool boundary(const Seqs& q, int32_t t, int32_t T) {
  if (t <= 0 || t >= T) return true;
  if (!q.cu) return false;
  return q.begin(q.of(t)) == t && q.of(t) > 0;
}

// 2^x h + e, of a whole segment: growing states may have a factor past float32's range and still be zero or small, so from 2^126 on
// it is taken in two halves (beyond 2^254 only denormal states would stay finite; theirs is taken as 2^254)
DEV float through(float x, float h, float e) {
  const bool large = x > 126.0f;
  const float f = hw_exp2(large ? fminf(0.5f * x, 127.0f) : x);
  return fmaf(f, large ? f * h : h, e);
}

// A state carried over `count` (at most K of them here) segments from segment s on, in steps of `dir`: the loads of all before
// the first is used
constexpr int BATCH = 8;
template <int NS, int K>
DEV void over_segments(const SsmArgs& p, const Where& w, int32_t s, int32_t count, int dir, int32_t d, int n0, const float (&A2)[NS],
                       float (&h)[NS]) {
  float e[K][NS], total[K];
  const int32_t D = static_cast<int32_t>(p.D);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int64_t at = (s + dir * (k < count ? k : count - 1)) * p.B + w.b;
    load_nd<NS>(p.end + at * p.D * p.N + d, D, p.N, n0, e[k]);
    total[k] = p.sum[at * p.D + d];
  }
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int n = 0; n < NS; ++n) h[n] = k < count ? through(A2[n] * total[k], h[n], e[k][n]) : h[n];
}

// ENDS: what each segment but the last leaves (from its last sequence's start, if one begins in it).  Otherwise the walk itself.
template <typename T, int NS, int WV, bool ENDS>
__global__ __launch_bounds__(WV * WAVE) void k_ssm(const SsmArgs p) {
  using L = Tile<T, NS, WV>;
  constexpr int E = L::E, NP = L::NP;
  __shared__ float2 u[CT][CH];
  __shared__ __attribute__((aligned(16))) float sb[CT * NP], sc[CT * NP];
  __shared__ float part[ENDS ? 1 : WV][CT][CH];
  __shared__ Marks marks;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Where w = where(p);
  const int32_t D_ = static_cast<int32_t>(p.D);
  const bool in = lane < w.left;
  const int32_t d = w.d + (in ? lane : w.left - 1);   // lanes past the last channel repeat it and store nothing
  const int n0 = wave * NS;
  const int64_t own = static_cast<int64_t>(d) * p.N;            // [d][N]
  const int64_t seq_step = p.D * p.N;                           // of h0 and h_last
  const int64_t row_states = w.b * p.seqs.n * seq_step + own;
  int32_t first = w.s * p.per, last = first + p.per < p.tiles ? first + p.per : p.tiles;   // tiles

  float A2[NS], h[NS] = {};
  load_dn<NS>(p.A + own, p.N, n0, A2);
#pragma unroll
  for (int n = 0; n < NS; ++n) A2[n] *= kLog2e;
  const float bias = in && p.dt_bias ? p.dt_bias[d] : 0.0f, skip = in && p.skip ? p.skip[d] : 0.0f;

  float sum = 0.0f;
  const int32_t ta = first * CT, tb = last * CT < p.T ? last * CT : p.T;
  int32_t begin = 0;            // ENDS: the segment's last start
  if constexpr (ENDS) {
    begin = p.seqs.cu ? static_cast<int32_t>(p.seqs.begin(p.seqs.of(tb - 1))) : 0;
    if (begin > ta) first = begin / CT;
  } else if (w.s > 0 && !boundary(p.seqs, ta, p.T)) {
    // the state entering: from the segment in which its sequence begins, over those between
    const int32_t from = p.seqs.cu ? static_cast<int32_t>(p.seqs.begin(p.seqs.of(ta))) : 0;
    int32_t s = from / (p.per * CT);
    const float* end = p.end + (s * p.B + w.b) * seq_step + d;
    load_nd<NS>(end, D_, p.N, n0, h);
    for (++s; s < w.s; s += BATCH) over_segments<NS, BATCH>(p, w, s, w.s - s, 1, d, n0, A2, h);
  }
  // the last sequence that begins in this segment: later segments' workgroups write over its h0 where that is h_last's place
  const int64_t last_seq = p.in_place && p.S > 1 ? p.seqs.of(tb - 1) : -1;

  Bits<T> x[E], dl[E], z[E], vb[L::BC], vc[L::BC];
  const int64_t from = static_cast<int64_t>(first) * CT;
  Column<T> cx(p.x, p.sx, w.b, from, w, lane), cd(p.delta, p.sdelta, w.b, from, w, lane), cz(p.z, p.sz, w.b, from, w, lane);
  Column<T> cy(p.y, p.sy, w.b, from, w, lane);
  Shared<T, NS, WV> cb(p.b, p.sb, w.b, from, w.g, p.N), cc(p.c, p.sc, w.b, from, w.g, p.N);
  float* carry = p.carry ? p.carry + (w.b * p.tiles + first) * seq_step + d : nullptr;
  const int32_t T_ = p.T, N = p.N;
  const bool gate = p.z;
  const auto load = [&](int32_t steps) {
    cx.load(wave, WV, steps, x);
    cd.load(wave, WV, steps, dl);
    cb.load(steps < CT ? steps : CT, vb);
    if constexpr (!ENDS) {
      if (gate) cz.load(wave, WV, steps, z);
      cc.load(steps < CT ? steps : CT, vc);
    }
  };
  load(T_ - first * CT);

  for (int32_t tile = first; tile < last; ++tile) {
    const int32_t t0 = tile * CT;
    const int32_t steps = T_ - t0 < CT ? T_ - t0 : CT;
    const auto* q = arguments<SsmArgs>();
    cx.s = q->sx[1], cd.s = q->sdelta[1], cb.s = q->sb[1];
    if constexpr (!ENDS) cz.s = q->sz[1], cc.s = q->sc[1], cy.s = q->sy[1];
    float xf[E], zf[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int t = wave + i * WV;
      xf[i] = value(x[i]);
      if constexpr (!ENDS) zf[i] = value(z[i]);
      const float dt = softplus(value(dl[i]) + bias);
      u[t][lane] = t < steps ? make_float2(dt, dt * xf[i]) : make_float2(0.0f, 0.0f);
    }
    Shared<T, NS, WV>::put(sb, vb);
    if constexpr (!ENDS) Shared<T, NS, WV>::put(sc, vc);
    __syncthreads();
    if (tile + 1 < last) {
      cx.move(CT);
      cd.move(CT);
      cb.move(CT);
      if constexpr (!ENDS) {
        cz.move(CT);
        cc.move(CT);
      }
      load(T_ - t0 - CT);
    }

    if constexpr (!ENDS) {
      if (carry) {
        store_nd<NS>(carry, D_, N, n0, in, h);
        carry += seq_step;
      }
    }
    const uint32_t starts = marks_of(p.seqs, t0, steps, marks);
    float rb[NS];
    get_shared<NS, NP>(sb, wave, lane, rb);
    // whole tiles in which no sequence begins are walked without a branch
    const auto walk = [&](auto events) {
      constexpr bool EVENTS = events;
      for_up<0, CT / 4>([&](auto quarter) {
        constexpr int Q = quarter * 4;
        if (!EVENTS || Q < steps) {
          for_up<Q, Q + 4>([&](auto step) {
            constexpr int t = step;
            if (EVENTS && t >= steps) return;     // exp(0 A) is no 1 for an infinite A
            if (EVENTS && (starts >> t & 1)) {
              if constexpr (ENDS) {
                if (t0 + t == begin) {
                  const int32_t j = p.seqs.cu ? uniform(marks.start[t]) : 0;
                  load_dn<NS>(p.h0 ? p.h0 + row_states + j * seq_step : nullptr, p.N, n0, h);
                  if (p.head) store_nd<NS>(p.head + (w.s * p.B + w.b) * seq_step + d, D_, p.N, n0, in, h);
                  sum = 0.0f;
                }
              } else {
                const auto* e = arguments<SsmArgs>();
                const int32_t j = e->seqs.cu ? uniform(marks.start[t]) : 0;
                if (t0 + t > ta && e->h_last)
                  store_dn<NS>(e->h_last + row_states + uniform(marks.before[t]) * seq_step, e->N, n0, in, h);
                if (j == last_seq && w.s + 1 < e->S)
                  load_nd<NS>(e->head + (w.s * e->B + w.b) * seq_step + d, D_, e->N, n0, h);
                else
                  load_dn<NS>(e->h0 ? e->h0 + row_states + j * seq_step : nullptr, e->N, n0, h);
              }
            }
            const float2 v = u[t][lane];
            if constexpr (ENDS) sum += v.x;
            float y = 0.0f, c[NS];
            if constexpr (!ENDS) step_values<NS, NP>(sc, wave, t, c);
            for_up<0, NS>([&](auto state) {
              constexpr int n = state;
              const float a = hw_exp2(A2[n] * v.x);
              h[n] = fmaf(a, h[n], of_step<NS, t, n>(rb) * v.y);
              if constexpr (!ENDS) y = n ? fmaf(c[n], h[n], y) : c[n] * h[n];
            });
            if constexpr (!ENDS) part[wave][t][lane] = y;
          });
        }
      });
    };
    if (steps < CT || (starts & kSteps)) walk(std::true_type{});
    else walk(std::false_type{});
    __syncthreads();
    if constexpr (!ENDS) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int t = wave + i * WV;
        float y = skip * xf[i];
#pragma unroll
        for (int k = 0; k < WV; ++k) y += part[k][t][lane];
        if (gate) y *= silu(zf[i]);
        if (t < steps && in) cy.store(t, y);
      }
      cy.move(CT);
    }
  }
  if constexpr (ENDS) {
    store_nd<NS>(p.end + (w.s * p.B + w.b) * seq_step + d, D_, p.N, n0, in, h);
    if (wave == 0 && in) p.sum[(w.s * p.B + w.b) * p.D + d] = sum;
  } else if (p.h_last) {
    // the sequence that ends with the segment, and with the row those that have no steps
    if (boundary(p.seqs, tb, p.T)) store_dn<NS>(p.h_last + row_states + p.seqs.of(tb - 1) * seq_step, p.N, n0, in, h);
    if (tb == p.T && p.seqs.cu && !p.in_place) {
      for (int64_t j0 = 0; j0 < p.seqs.n; j0 += WAVE) {
        const int64_t j = j0 + lane;
        uint64_t empty = __builtin_amdgcn_ballot_w64(j < p.seqs.n && p.seqs.end(j) <= p.seqs.begin(j));
        for (; empty; empty &= empty - 1) {
          const int64_t at = (j0 + __builtin_ctzll(empty)) * seq_step;
          float v[NS];
          load_dn<NS>(p.h0 ? p.h0 + row_states + at : nullptr, p.N, n0, v);
          store_dn<NS>(p.h_last + row_states + at, p.N, n0, in, v);
        }
      }
    }
  }
}

// ------------------------------------------------------------------------------------------------
// Few steps (kSerial or fewer, one generated token for instance): WV lanes a channel, NS states a lane, all steps in order, no
// shared memory, one launch.  A channel's states are read as they lie, [d][N], by neighbouring lanes.  Sums are formed as the
// tiles form them: the same bits.  Bound by the launch and one round trip to memory.
// ------------------------------------------------------------------------------------------------
constexpr int32_t kSerial = 8;   // T = 1, 4, 8, 12: 5.2, 7.5, 10.8, 13.9 us against the tiles' 12.6, 12.5, 12.9, 13.6 (B = 32, D = 2048, N = 16, bf16)
template <typename T, int NS, int WV>
__global__ __launch_bounds__(256) void k_ssm_serial(const SsmArgs p, int64_t lanes) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const bool there = id < lanes;
  const int64_t at = there ? id : lanes - 1, cell = at / WV;
  const int part = static_cast<int>(at - cell * WV), n0 = part * NS, base = (threadIdx.x & 63) - part;
  const int64_t b = cell / p.D, d = cell - b * p.D, g = d / p.group;
  const bool first = there && part == 0;
  float A2[NS], h[NS];
  const int64_t own = d * p.N, seq_step = p.D * p.N, row = b * p.seqs.n * seq_step + own;
  load_dn<NS>(p.A + own, p.N, n0, A2);
#pragma unroll
  for (int n = 0; n < NS; ++n) A2[n] *= kLog2e;
  const float bias = p.dt_bias ? p.dt_bias[d] : 0.0f, skip = p.skip ? p.skip[d] : 0.0f;
  int64_t t = 0;
  for (int64_t j = 0; j < p.seqs.n; ++j) {
    const int64_t stop = p.seqs.end(j);
    load_dn<NS>(p.h0 ? p.h0 + row + j * seq_step : nullptr, p.N, n0, h);
    for (; t < stop; ++t) {
      if (t == 0 && p.carry) store_nd<NS>(p.carry + b * seq_step + d, static_cast<int32_t>(p.D), p.N, n0, there, h);
      const float x = to_f32(static_cast<const T*>(p.x)[b * p.sx[0] + t * p.sx[1] + d]);
      const float dt = softplus(to_f32(static_cast<const T*>(p.delta)[b * p.sdelta[0] + t * p.sdelta[1] + d]) + bias);
      const T* pb = static_cast<const T*>(p.b) + b * p.sb[0] + t * p.sb[1] + g * p.sb[2];
      const T* pc = static_cast<const T*>(p.c) + b * p.sc[0] + t * p.sc[1] + g * p.sc[2];
      float vb[NS], vc[NS];
      if constexpr (NS == 1) {
        vb[0] = to_f32(*pb), vc[0] = to_f32(*pc);
      } else {
        const Vec<T, NS> rb = load_row<T, NS>(pb + n0, p.N - n0, T{}), rc = load_row<T, NS>(pc + n0, p.N - n0, T{});
#pragma unroll
        for (int n = 0; n < NS; ++n) vb[n] = rb.get(n), vc[n] = rc.get(n);
      }
      const float u = dt * x;
      float y = 0.0f;
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        h[n] = fmaf(hw_exp2(A2[n] * dt), h[n], vb[n] * u);
        y = n ? fmaf(vc[n], h[n], y) : vc[n] * h[n];
      }
      float sum = skip * x;
#pragma unroll
      for (int k = 0; k < WV; ++k) sum += __shfl(y, base + k);
      if (p.z) sum *= silu(to_f32(static_cast<const T*>(p.z)[b * p.sz[0] + t * p.sz[1] + d]));
      if (first) static_cast<T*>(p.y)[b * p.sy[0] + t * p.sy[1] + d] = from_f32<T>(sum);
    }
    if (p.h_last) store_dn<NS>(p.h_last + row + j * seq_step, p.N, n0, there, h);
  }
}

// no steps: every state leaves as it came (rest: where d_last becomes d_h0)
__global__ __launch_bounds__(256) void k_copy_states(const float* from, float* to, int64_t n) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) to[i] = from ? from[i] : 0.0f;
}

// ------------------------------------------------------------------------------------------------
// Gradients.  With G_t = dL/dy_t z sig(z) (G = dL/dy without a gate), q_t = dL/dh_t = C_t G_t + P_t, P_{t-1} = a_t q_t (plus d_last
// at a sequence's last step) and e_t = P_{t-1} h_{t-1}:
//   d(dt x) = sum_n q B,  d(dt) += sum_n e A,  d_A = sum_t e dt,  d_B = sum_d q dt x,  d_C = sum_d G h.
// A tile's states are rebuilt from the carry and stay, with their decays, in registers; the way back walks them in reverse.  The
// sums over states go through shared memory as y's do.  Those over channels are formed for 32 values at a time (two for
// each step and state): halves, rows, half rows and quads of the wave are folded onto each other, each time leaving half the
// registers, so a value costs two instructions and not six.  Each channel tile's sums go to the workspace, and one launch more
// adds them up.  Segments as in the forward pass, from the right.
// ------------------------------------------------------------------------------------------------
template <int TO, int FROM, typename F> DEV void for_down(F&& f) {   // FROM - 1 .. TO
  if constexpr (FROM > TO) {
    f(Int<FROM - 1>{});
    for_down<TO, FROM - 1>(f);
  }
}

// Sums over the wave's lanes of 32 values; lane l gets that of value 16 l5 + 8 l4 + 4 l3 + 2 l2 + l0 (l5: bit 5 of l)
DEV float fold(float (&v)[32], int lane) {
  for_up<0, 16>([&](auto k) {
    constexpr int i = k;
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[i]), __float_as_uint(v[i + 16]), false, false);
    v[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  });
  for_up<0, 8>([&](auto k) {
    constexpr int i = k;
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[i]), __float_as_uint(v[i + 8]), false, false);
    v[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  });
  for_up<0, 4>([&](auto k) {
    constexpr int i = k;
    const float a = v[i] + dpp<0x128>(v[i]), b = v[i + 4] + dpp<0x128>(v[i + 4]);   // row_ror:8
    v[i] = lane & 8 ? b : a;
  });
  for_up<0, 2>([&](auto k) {
    constexpr int i = k;
    const float a = v[i] + dpp<0x141>(v[i]), b = v[i + 2] + dpp<0x141>(v[i + 2]);   // row_half_mirror
    v[i] = lane & 4 ? b : a;
  });
  for_up<0, 2>([&](auto k) {
    constexpr int i = k;
    v[i] += dpp<0xb1>(v[i]);
    v[i] += dpp<0x4e>(v[i]);
  });
  return lane & 1 ? v[1] : v[0];
}

// What flows out of each segment but the first to the steps before it, if nothing enters it from the right, and the sum of dt over
// the steps that it flows through
template <typename T, int NS, int WV>
__global__ __launch_bounds__(WV * WAVE) void k_ssm_back_ends(const SsmGradArgs g) {
  const SsmArgs& p = g.f;
  using L = Tile<T, NS, WV>;
  constexpr int E = L::E, NP = L::NP;
  __shared__ float2 u[CT][CH];
  __shared__ __attribute__((aligned(16))) float sc[CT * NP];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Where w = where(p);
  ++w.s;
  const int32_t D_ = static_cast<int32_t>(p.D);
  const bool in = lane < w.left;
  const int32_t d = w.d + (in ? lane : w.left - 1);   // lanes past the last channel repeat it and store nothing
  const int n0 = wave * NS;
  const int64_t seq_step = p.D * p.N, own = static_cast<int64_t>(d) * p.N;
  const int32_t first = w.s * p.per, last = first + p.per < p.tiles ? first + p.per : p.tiles;
  const int32_t ta = first * CT, tb = last * CT < p.T ? last * CT : p.T;
  // the steps [ta, end) of the sequence that ta belongs to
  const int64_t j = p.seqs.cu ? p.seqs.of(ta) : 0;
  int32_t stop = static_cast<int32_t>(p.seqs.end(j));
  stop = stop > ta ? stop : ta + 1;
  const int32_t end = stop < tb ? stop : tb;

  float A2[NS], P[NS] = {}, sum = 0.0f;
  load_dn<NS>(p.A + own, p.N, n0, A2);
#pragma unroll
  for (int n = 0; n < NS; ++n) A2[n] *= kLog2e;
  const float bias = in && p.dt_bias ? p.dt_bias[d] : 0.0f;
  if (stop <= tb) load_dn<NS>(g.d_last ? g.d_last + (w.b * p.seqs.n + j) * seq_step + own : nullptr, p.N, n0, P);

  Bits<T> dl[E], z[E], dy[E], vc[L::BC];
  int32_t tile = (end - 1) / CT;
  const int64_t from = static_cast<int64_t>(tile) * CT;
  Column<T> cd(p.delta, p.sdelta, w.b, from, w, lane), cz(p.z, p.sz, w.b, from, w, lane), cg(g.dy, g.sdy, w.b, from, w, lane);
  Shared<T, NS, WV> cc(p.c, p.sc, w.b, from, w.g, p.N);
  const bool gate = p.z;
  const auto load = [&](int32_t steps) {
    cd.load(wave, WV, steps, dl);
    cg.load(wave, WV, steps, dy);
    if (gate) cz.load(wave, WV, steps, z);
    cc.load(steps < CT ? steps : CT, vc);
  };
  load(end - tile * CT);
  for (; tile >= first; --tile) {
    const int32_t t0 = tile * CT, steps = end - t0 < CT ? end - t0 : CT;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int t = wave + i * WV;
      float G = value(dy[i]);
      if (gate) G *= silu(value(z[i]));
      u[t][lane] = t < steps ? make_float2(softplus(value(dl[i]) + bias), G) : make_float2(0.0f, 0.0f);
    }
    Shared<T, NS, WV>::put(sc, vc);
    __syncthreads();
    if (tile > first) {
      cd.move(-CT);
      cz.move(-CT);
      cg.move(-CT);
      cc.move(-CT);
      load(CT);
    }
    const auto walk = [&](auto whole) {
      for_down<0, CT / 4>([&](auto quarter) {
        constexpr int Q = quarter * 4;
        if (whole || Q < steps) {
          for_down<Q, Q + 4>([&](auto step) {
            constexpr int t = step;
            if (!whole && t >= steps) return;     // exp(0 A) is no 1 for an infinite A
            const float2 v = u[t][lane];
            float c[NS];
            step_values<NS, NP>(sc, wave, t, c);
            sum += v.x;
            for_up<0, NS>([&](auto state) {
              constexpr int n = state;
              P[n] = hw_exp2(A2[n] * v.x) * fmaf(c[n], v.y, P[n]);
            });
          });
        }
      });
    };
    if (steps < CT) walk(std::false_type{});
    else walk(std::true_type{});
    __syncthreads();
  }
  store_nd<NS>(p.end + (w.s * p.B + w.b) * seq_step + d, D_, p.N, n0, in, P);
  if (wave == 0 && in) p.sum[(w.s * p.B + w.b) * p.D + d] = sum;
}

template <typename T, int NS, int WV>
__global__ __launch_bounds__(WV * WAVE, 2) void k_ssm_back(const SsmGradArgs g) {
  const SsmArgs& p = g.f;
  using L = Tile<T, NS, WV>;
  constexpr int E = L::E, NP = L::NP;
  constexpr int HT = CT / 2, RS = HT * NS < 16 ? HT : 16 / NS;   // steps of a half tile, and of those whose sums are formed at once
  __shared__ float2 u[CT][CH];
  __shared__ float sg[CT][CH];
  __shared__ __attribute__((aligned(16))) float sb[CT * NP], sc[CT * NP];
  __shared__ float part[3][WV][CT][CH];
  __shared__ Marks marks;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Where w = where(p);
  const int32_t D_ = static_cast<int32_t>(p.D);
  const bool in = lane < w.left;
  const int32_t d = w.d + (in ? lane : w.left - 1);   // lanes past the last channel repeat it and store nothing
  const int n0 = wave * NS;
  const int64_t seq_step = p.D * p.N, own = static_cast<int64_t>(d) * p.N;
  const int64_t row_states = w.b * p.seqs.n * seq_step + own;
  const int32_t first = w.s * p.per, last = first + p.per < p.tiles ? first + p.per : p.tiles;
  const int32_t tb = last * CT < p.T ? last * CT : p.T;

  // lanes past the last channel have rates and states of zero, like their steps: 0 NaN would enter the sums over channels
  float A2[NS], P[NS] = {}, dA[NS] = {}, d_skip = 0.0f, d_bias = 0.0f;
  load_dn<NS>(p.A + own, p.N, n0, A2);
  const auto inside = [&](float (&v)[NS]) {
#pragma unroll
    for (int n = 0; n < NS; ++n) v[n] = in ? v[n] : 0.0f;
  };
  inside(A2);
#pragma unroll
  for (int n = 0; n < NS; ++n) A2[n] *= kLog2e;
  const float bias = in && p.dt_bias ? p.dt_bias[d] : 0.0f, skip = in && p.skip ? p.skip[d] : 0.0f;
  if (!boundary(p.seqs, tb, p.T)) {
    // what enters from the right: from the segment that the sequence ends in, over those between
    int32_t stop = p.seqs.cu ? static_cast<int32_t>(p.seqs.end(p.seqs.of(tb))) : p.T;
    stop = stop > tb ? stop : tb + 1;
    int32_t s = (stop - 1) / (p.per * CT);
    load_nd<NS>(p.end + (s * p.B + w.b) * seq_step + d, D_, p.N, n0, P);
    for (--s; s > w.s; s -= BATCH) over_segments<NS, BATCH>(p, w, s, s - w.s, -1, d, n0, A2, P);
    inside(P);
  }

  Bits<T> x[E], dl[E], z[E], dy[E], vb[L::BC], vc[L::BC];
  float h_in[NS];
  const int64_t from = static_cast<int64_t>(last - 1) * CT;
  Column<T> cx(p.x, p.sx, w.b, from, w, lane), cd(p.delta, p.sdelta, w.b, from, w, lane), cz(p.z, p.sz, w.b, from, w, lane),
      cg(g.dy, g.sdy, w.b, from, w, lane);
  Column<T> ox(g.dx, g.sdx, w.b, from, w, lane), od(g.ddelta, g.sddelta, w.b, from, w, lane), oz(g.dz, g.sdz, w.b, from, w, lane);
  Shared<T, NS, WV> cb(p.b, p.sb, w.b, from, w.g, p.N), cc(p.c, p.sc, w.b, from, w.g, p.N);
  const float* carry = g.carry + (w.b * p.tiles + last - 1) * seq_step + d;
  const int32_t T_ = p.T, N = p.N;
  const bool gate = p.z;
  const auto load = [&](int32_t steps) {
    cx.load(wave, WV, steps, x);
    cd.load(wave, WV, steps, dl);
    cg.load(wave, WV, steps, dy);
    if (gate) cz.load(wave, WV, steps, z);
    cb.load(steps < CT ? steps : CT, vb);
    cc.load(steps < CT ? steps : CT, vc);
    load_nd<NS>(carry, D_, N, n0, h_in);
  };
  load(T_ - (last - 1) * CT);
  // where this lane's channel sums of a tile go
  const int fk = (lane & 1) | (lane >> 1 & 14), ft = fk / NS, fn = n0 + fk % NS;
  const bool sums = !(lane & 2) && fk < RS * NS && fn < N;
  float* bc = g.part_bc + ((static_cast<int64_t>(w.ct) * p.B + w.b) * T_ + from + ft) * (2 * N) + (lane >> 5) * N + fn;

  for (int32_t tile = last - 1; tile >= first; --tile) {
    const int32_t t0 = tile * CT, steps = T_ - t0 < CT ? T_ - t0 : CT;
    const auto* q = arguments<SsmGradArgs>();
    cx.s = q->f.sx[1], cd.s = q->f.sdelta[1], cz.s = q->f.sz[1], cg.s = q->sdy[1], cb.s = q->f.sb[1], cc.s = q->f.sc[1];
    ox.s = q->sdx[1], od.s = q->sddelta[1], oz.s = q->sdz[1];
    float xf[E], zf[E], dyf[E], open[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int t = wave + i * WV;
      const bool there = t < steps && in;      // what other lanes hold must not enter the sums over channels
      xf[i] = value(x[i]);
      zf[i] = gate ? value(z[i]) : 0.0f;
      dyf[i] = value(dy[i]);
      const float raw = value(dl[i]) + bias, dt = softplus(raw);
      open[i] = sigmoid(raw);
      u[t][lane] = there ? make_float2(dt, dt * xf[i]) : make_float2(0.0f, 0.0f);
      sg[t][lane] = there ? dyf[i] * (gate ? silu(zf[i]) : 1.0f) : 0.0f;
    }
    Shared<T, NS, WV>::put(sb, vb);
    Shared<T, NS, WV>::put(sc, vc);
    float h0[NS];
#pragma unroll
    for (int n = 0; n < NS; ++n) h0[n] = in ? h_in[n] : 0.0f;
    __syncthreads();
    if (tile > first) {
      cx.move(-CT);
      cd.move(-CT);
      cg.move(-CT);
      cz.move(-CT);
      cb.move(-CT);
      cc.move(-CT);
      carry -= seq_step;
      load(CT);
    }

    const uint32_t starts = marks_of(p.seqs, t0, steps, marks);
    const uint32_t ends = (starts & kSteps) >> 1 | (starts >> CT & 1) << (steps - 1);
    const auto entering = [&](int t, float (&v)[NS]) {          // the state entering the sequence that begins at step t
      const auto* e = arguments<SsmGradArgs>();
      const int32_t j = e->f.seqs.cu ? uniform(marks.start[t]) : 0;
      load_dn<NS>(e->f.h0 ? e->f.h0 + row_states + j * seq_step : nullptr, e->f.N, n0, v);
      inside(v);
    };
    float rb[NS], tA[NS] = {}, hm[NS];
    get_shared<NS, NP>(sb, wave, lane, rb);
    // the state between the halves of the tile
    for_up<0, NS>([&](auto state) { hm[state] = h0[state]; });
    const auto middle = [&](auto events) {
      for_up<0, HT>([&](auto step) {
        constexpr int t = step;
        if (events && (starts >> t & 1)) entering(t, hm);
        const float2 v = u[t][lane];
        for_up<0, NS>([&](auto state) {
          constexpr int n = state;
          hm[n] = fmaf(hw_exp2(A2[n] * v.x), hm[n], of_step<NS, t, n>(rb) * v.y);
        });
      });
    };
    const auto back = [&](auto events, const int half) {
      const int s0 = half * HT;
      const uint32_t here = starts >> s0, over = ends >> s0;   // (the bit past the tile is asked for by no step)
      float hb[NS], hi[NS], hs[HT][NS], as[HT][NS];
      for_up<0, NS>([&](auto state) {
        constexpr int n = state;
        hi[n] = half ? hm[n] : h0[n];
        if constexpr (NS > 1) {
          hb[n] = half ? rb[(n + NS / 2) % NS] : rb[n];
        } else {
          hb[0] = half ? dpp<0x128>(rb[0]) : rb[0];   // row_ror:8
        }
      });
      for_up<0, HT>([&](auto step) {
        constexpr int t = step;
        float h[NS], y = 0.0f;
        for_up<0, NS>([&](auto state) { h[state] = t == 0 ? hi[state] : hs[t == 0 ? 0 : t - 1][state]; });
        if (events && (here >> t & 1)) entering(s0 + t, h);
        const float2 v = u[s0 + t][lane];
        float c[NS];
        step_values<NS, NP>(sc, wave, s0 + t, c);
        const bool past = events && s0 + t >= steps;            // exp(0 A) is no 1 for an infinite A
        for_up<0, NS>([&](auto state) {
          constexpr int n = state;
          as[t][n] = past ? 1.0f : hw_exp2(A2[n] * v.x);
          hs[t][n] = fmaf(as[t][n], h[n], of_step<NS, t, n>(hb) * v.y);
          y = n ? fmaf(c[n], hs[t][n], y) : c[n] * hs[t][n];
        });
        part[0][wave][s0 + t][lane] = y;
      });
      for_down<0, HT / RS>([&](auto block) {
        constexpr int Q = block * RS;
        float v32[32];
        if constexpr (RS * NS < 16) for_up<0, 32>([&](auto i) { v32[i] = 0.0f; });
        for_down<Q, Q + RS>([&](auto step) {
          constexpr int t = step;
          if (events && (over >> t & 1)) {
            const auto* e = arguments<SsmGradArgs>();
            const int32_t j = e->f.seqs.cu ? uniform(marks.before[s0 + t + 1]) : 0;
            load_dn<NS>(e->d_last ? e->d_last + row_states + j * seq_step : nullptr, e->f.N, n0, P);
            inside(P);
          }
          const float2 v = u[s0 + t][lane];
          const float G = sg[s0 + t][lane];
          float h[NS], b[NS], c[NS], s1 = 0.0f, s2 = 0.0f;
          step_values<NS, NP>(sb, wave, s0 + t, b);
          step_values<NS, NP>(sc, wave, s0 + t, c);
          for_up<0, NS>([&](auto state) { h[state] = t == 0 ? hi[state] : hs[t == 0 ? 0 : t - 1][state]; });
          if (events && (here >> t & 1)) entering(s0 + t, h);
          for_up<0, NS>([&](auto state) {
            constexpr int n = state;
            const float q = fmaf(c[n], G, P[n]);
            s1 = n ? fmaf(b[n], q, s1) : b[n] * q;
            v32[(t - Q) * NS + n] = q * v.y;
            v32[16 + (t - Q) * NS + n] = G * hs[t][n];
            P[n] = as[t][n] * q;
            const float e = P[n] * h[n];
            s2 = n ? fmaf(e, A2[n], s2) : e * A2[n];
            tA[n] = fmaf(e, v.x, tA[n]);
          });
          part[1][wave][s0 + t][lane] = s1;
          part[2][wave][s0 + t][lane] = s2;
          if (events && (here >> t & 1)) {
            const auto* e = arguments<SsmGradArgs>();
            const int32_t j = e->f.seqs.cu ? uniform(marks.start[s0 + t]) : 0;
            if (e->d_h0) store_dn<NS>(e->d_h0 + row_states + j * seq_step, e->f.N, n0, in, P);
          }
        });
        const float sum = fold(v32, lane);
        if (sums && s0 + Q + ft < steps) bc[(s0 + Q) * (2 * N)] = sum;
      });
    };
    // tiles in which no sequence begins or ends are walked without a branch
    if (starts) {
      if (steps > HT) middle(std::true_type{});
#pragma unroll 1
      for (int half = steps > HT ? 1 : 0; half >= 0; --half) back(std::true_type{}, half);
    } else {
      middle(std::false_type{});
#pragma unroll 1
      for (int half = 1; half >= 0; --half) back(std::false_type{}, half);
    }
#pragma unroll
    for (int n = 0; n < NS; ++n) dA[n] += tA[n];
    __syncthreads();
    float tskip = 0.0f, tbias = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int t = wave + i * WV;
      if (t < steps) {
        float y = skip * xf[i], s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int k = 0; k < WV; ++k) {
          y += part[0][k][t][lane];
          s1 += part[1][k][t][lane];
          s2 += part[2][k][t][lane];
        }
        const float dt = u[t][lane].x, G = sg[t][lane];
        const float dd = fmaf(s1, xf[i], kLn2 * s2) * open[i];   // s2 is of A log2(e)
        tskip = fmaf(G, xf[i], tskip);
        tbias += dd;
        if (in) {
          ox.store(t, fmaf(s1, dt, G * skip));
          od.store(t, dd);
          if (gate) oz.store(t, dyf[i] * y * silu_slope(zf[i], sigmoid(zf[i])));
        }
      }
    }
    ox.move(-CT);
    od.move(-CT);
    oz.move(-CT);
    bc -= static_cast<int64_t>(CT) * (2 * N);
    d_skip += tskip;
    d_bias += tbias;
    __syncthreads();            // u and sg are read above
  }

  // parameters: [S B][N + 2][D]
  const int64_t row = (w.s * p.B + w.b) * static_cast<int64_t>(p.N + 2) * p.D + d;
  store_nd<NS>(g.part_A + row, D_, p.N, n0, in, dA);
  part[0][wave][0][lane] = d_skip;
  part[0][wave][1][lane] = d_bias;
  __syncthreads();
  if (wave == 0 && in) {
    float s = 0.0f, b = 0.0f;
#pragma unroll
    for (int k = 0; k < WV; ++k) {
      s += part[0][k][0][lane];
      b += part[0][k][1][lane];
    }
    g.part_A[row + p.N * p.D] = s;
    g.part_A[row + (p.N + 1) * p.D] = b;
  }
}

// d_b and d_c: a thread adds up the channel tiles' sums of one group for one value
struct SharedArgs {
  const float* part;
  int64_t B, T;
  int32_t N, G, ctiles;
  void *db, *dc;
  int64_t sdb[3], sdc[3];
};
template <typename T> __global__ __launch_bounds__(256) void k_ssm_shared(const SharedArgs p) {
  const int64_t plane = p.B * p.T * (2 * p.N), id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (id >= plane * p.G) return;
  const int64_t g = id / plane, e = id - g * plane, row = e / (2 * p.N), b = row / p.T, t = row - b * p.T;
  const int32_t k = static_cast<int32_t>(e - row * (2 * p.N));
  const float* from = p.part + g * p.ctiles * plane + e;
  float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
  int32_t c = 0;
  for (; c + 4 <= p.ctiles; c += 4, from += 4 * plane) {
    s0 += from[0];
    s1 += from[plane];
    s2 += from[2 * plane];
    s3 += from[3 * plane];
  }
  for (; c < p.ctiles; ++c, from += plane) s0 += *from;
  const float s = (s0 + s1) + (s2 + s3);
  if (k < p.N) static_cast<T*>(p.db)[b * p.sdb[0] + t * p.sdb[1] + g * p.sdb[2] + k] = from_f32<T>(s);
  else static_cast<T*>(p.dc)[b * p.sdc[0] + t * p.sdc[1] + g * p.sdc[2] + k - p.N] = from_f32<T>(s);
}
// where the column sums [N + 2][D] go: d_A [D][N], d_skip and d_dt_bias [D]
struct ToParams {
  int64_t D;
  int32_t N;
  float *d_A, *d_skip, *d_bias;
  DEV void operator()(int64_t, int64_t i, float v) const {
    const int64_t n = i / D, d = i - n * D;
    float* to = n < N ? d_A : n == N ? d_skip : d_bias;
    if (to) to[n < N ? d * N + n : d] = v;
  }
};
// d_h0 of sequences without steps
__global__ __launch_bounds__(256) void k_ssm_empty(const Seqs q, int64_t states, int64_t n, const float* d_last, float* d_h0) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n) return;
  const int64_t j = i / states % q.n;
  if (q.end(j) <= q.begin(j)) d_h0[i] = d_last ? d_last[i] : 0.0f;
}

// ---------------- host ----------------
struct Split {
  int64_t ctiles, tiles, rows;   // channel tiles of a group, tiles of a row, workgroups without segments
  int64_t S, per;
};
// Segments of a row: as many as bring `want` workgroups, each of at least kLeast tiles, where those without fill less than the chip
// holds at a time.  bf16, N = 16, forward and gradient: B = 8, T = 2048, D = 2048 (256 workgroups) 228 and 593 us against 284 and 782
// whole; B = 16 (512) 412 and 1155 against 353 and 1046.
constexpr int64_t kFull = 448, kWant = 2048, kGradWant = 1536, kLeast = 2, kMost = 96;
static Split split(int64_t B, int64_t T, int64_t D, int64_t G, int64_t want) {
  Split s;
  if (D == 0) G = 1;
  s.ctiles = ceil_div(D / G, CH);
  s.tiles = ceil_div(T, CT);
  s.rows = B * G * s.ctiles;
  int64_t n = 1;
  if (s.rows && s.rows < kFull) n = want / s.rows;
  if (n > s.tiles / kLeast) n = s.tiles / kLeast;
  if (n > kMost) n = kMost;     // each is entered over those before it
  if (n < 1) n = 1;
  s.per = s.tiles ? ceil_div(s.tiles, n) : 1;
  s.S = s.tiles ? ceil_div(s.tiles, s.per) : 1;
  return s;
}
static Split forward_split(int64_t B, int64_t T, int64_t D, int64_t G) { return split(B, T, D, G, kWant); }
static Split gradient_split(int64_t B, int64_t T, int64_t D, int64_t G) { return split(B, T, D, G, kGradWant); }

static bool sizes_ok(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G) {
  if (N < 1 || N > INT64_MAX / 128 || G < 1 || G > INT32_MAX || !sizes_fit(B, T, D) || (D > 0 && (G > D || D % G))) return false;
  if (D == 0) G = 1;            // no channels: any number of groups
  return sizes_fit(D, N + 2) && sizes_fit(B, ceil_div(T, CT) + 1, D) &&
         (D == 0 || B == 0 || N + 2 <= INT64_MAX / 64 / (D * B) / (ceil_div(T, CT) + 1)) &&
         (B == 0 || T == 0 || N <= INT64_MAX / 64 / B / T / (D / 64 + G + 1));
}
struct Room {   // floats: the segments' parts, then (gradient) the sums
  int64_t end, sum, head, bc, part, scratch;
  int64_t total() const { return end + sum + head + bc + part + scratch; }
};
static int64_t round64(int64_t n) { return ceil_div(n, 64) * 64; }
static Room room(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G, bool gradient) {
  const Split s = gradient ? gradient_split(B, T, D, G) : forward_split(B, T, D, G);
  Room r{};
  if (s.S > 1) {
    r.end = round64(s.S * B * N * D);
    r.sum = round64(s.S * B * D);
    if (!gradient) r.head = r.end;
  }
  if (gradient) {
    const int64_t rows = T ? s.S * B : 0;
    r.bc = round64(G * s.ctiles * B * T * 2 * N);
    r.part = round64(rows * (N + 2) * D);
    r.scratch = round64(colsum_floats(rows, (N + 2) * D));
  }
  return r;
}

static bool problem_ok(const pararnn_block_ssm* q) {
  if (!q || !dtype_ok(q->dtype) || !sizes_ok(q->B, q->T, q->D, q->N, q->G)) return false;
  const size_t e = dtype_size(q->dtype);
  const bool any = q->B > 0 && q->D > 0, steps = any && q->T > 0;
  if (!ptr_ok(q->x, e, steps) || !ptr_ok(q->delta, e, steps) || !ptr_ok(q->z, e, false) || !ptr_ok(q->b, e, steps) ||
      !ptr_ok(q->c, e, steps) || !ptr_ok(q->A, 4, any) || !ptr_ok(q->skip, 4, false) || !ptr_ok(q->dt_bias, 4, false) ||
      !ptr_ok(q->h0, 4, false) || !ptr_ok(q->cu_seqlens, 4, false))
    return false;
  if (q->cu_seqlens) {
    if (q->n_seqs < 1 || q->T > INT32_MAX || !sizes_fit(q->B, q->n_seqs, q->D)) return false;
    if (any && q->N > INT64_MAX / 16 / (q->B * q->n_seqs * q->D)) return false;
  }
  const int64_t(*s2[3])[2] = {&q->sx, &q->sdelta, &q->sz};
  for (int k = 0; k < (q->z ? 3 : 2); ++k)
    if (!plane_ok(q->B, (*s2[k])[0]) || !plane_ok(q->T, (*s2[k])[1])) return false;
  const int64_t(*s3[2])[3] = {&q->sb, &q->sc};
  for (const auto* s : s3)
    if (!plane_ok(q->B, (*s)[0]) || !plane_ok(q->T, (*s)[1]) || !plane_ok(q->G, (*s)[2])) return false;
  return true;
}
// A step's stride as the kernels take it: that of a single step means nothing, and is any number.
static int64_t step_of(const pararnn_block_ssm* q, int64_t stride) { return q->T > 1 ? stride : 0; }
// a step's stride that does not fit the offsets inside a tile
static bool far(const pararnn_block_ssm* q, int64_t stride) { return step_of(q, stride) >= PARARNN_BLOCK_SSM_MAX_STEP; }
static bool supported(const pararnn_block_ssm* q, const Split& s, int threads) {
  if (far(q, q->sx[1]) || far(q, q->sdelta[1]) || (q->z && far(q, q->sz[1])) || far(q, q->sb[1]) || far(q, q->sc[1])) return false;
  if (q->N > PARARNN_BLOCK_MAX_STATES || q->T > INT32_MAX - CT || q->D > INT32_MAX / 64) return false;
  if (s.ctiles * q->G > INT32_MAX || q->B > INT32_MAX) return false;
  return s.rows == 0 || (s.S <= INT64_C(0xffffffff) / s.rows && grid_ok(s.rows * s.S, threads));
}
static SsmArgs ssm_args(const pararnn_block_ssm* q, const Split& s) {
  SsmArgs p{};
  p.x = q->x, p.delta = q->delta, p.z = q->z, p.b = q->b, p.c = q->c;
  for (int k = 0; k < 2; ++k) p.sx[k] = q->sx[k], p.sdelta[k] = q->sdelta[k], p.sz[k] = q->sz[k];
  for (int k = 0; k < 3; ++k) p.sb[k] = q->sb[k], p.sc[k] = q->sc[k];
  for (int64_t* t : {&p.sx[1], &p.sdelta[1], &p.sz[1], &p.sb[1], &p.sc[1]}) *t = step_of(q, *t);
  p.A = q->A, p.skip = q->skip, p.dt_bias = q->dt_bias, p.h0 = q->h0;
  p.seqs = {q->cu_seqlens, q->cu_seqlens ? q->n_seqs : 1, q->T};
  p.B = q->B, p.D = q->D;
  p.T = static_cast<int32_t>(q->T), p.N = static_cast<int32_t>(q->N), p.G = static_cast<int32_t>(q->G);
  p.tiles = static_cast<int32_t>(s.tiles);
  p.ctiles = static_cast<int32_t>(s.ctiles), p.group = static_cast<int32_t>(q->D / q->G);
  p.S = static_cast<int32_t>(s.S), p.per = static_cast<int32_t>(s.per);
  return p;
}

template <typename T, int NS, int WV> struct Forward {
  static pararnn_status run(const SsmArgs& p, const Split& s, hipStream_t st) {
    const int64_t lanes = p.B * p.D * WV, blocks = ceil_div(lanes, 256);
    if (p.T <= kSerial && grid_ok(blocks, 256)) {
      k_ssm_serial<T, NS, WV><<<dim3(static_cast<uint32_t>(blocks)), dim3(256), 0, st>>>(p, lanes);
      return launched();
    }
    if (s.S > 1)
      k_ssm<T, NS, WV, true><<<dim3(static_cast<uint32_t>(s.rows * (s.S - 1))), dim3(WV * WAVE), 0, st>>>(p);
    k_ssm<T, NS, WV, false><<<dim3(static_cast<uint32_t>(s.rows * s.S)), dim3(WV * WAVE), 0, st>>>(p);
    return launched();
  }
};
template <typename T, int NS, int WV> struct Backward {
  static pararnn_status run(const SsmGradArgs& g, const Split& s, hipStream_t st) {
    if (s.S > 1) k_ssm_back_ends<T, NS, WV><<<dim3(static_cast<uint32_t>(s.rows * (s.S - 1))), dim3(WV * WAVE), 0, st>>>(g);
    k_ssm_back<T, NS, WV><<<dim3(static_cast<uint32_t>(s.rows * s.S)), dim3(WV * WAVE), 0, st>>>(g);
    return launched();
  }
};
// waves of a workgroup for N states: four states a wave, two for up to four (one wave would load a tile by itself, and spill)
static int waves_of(int64_t N) { return N == 1 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : 8; }
template <template <typename, int, int> class F, typename T, typename A>
static pararnn_status by_states(int64_t N, const A& a, const Split& s, hipStream_t st) {
  if (N == 1) return F<T, 1, 1>::run(a, s, st);
  if (N <= 4) return F<T, 2, 2>::run(a, s, st);
  switch (waves_of(N)) {
    case 2: return F<T, 4, 2>::run(a, s, st);
    case 4: return F<T, 4, 4>::run(a, s, st);
    default: return F<T, 4, 8>::run(a, s, st);
  }
}

}  // namespace lm

using namespace lm;

extern "C" int64_t pararnn_block_ssm_chunks(int64_t T) { return T < 0 ? 0 : ceil_div(T, CT); }

extern "C" size_t pararnn_block_ssm_workspace_bytes(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G, int gradient) {
  if (!sizes_ok(B, T, D, N, G) || N > PARARNN_BLOCK_MAX_STATES) return 0;
  return static_cast<size_t>(room(B, T, D, N, G, gradient != 0).total()) * sizeof(float);
}

extern "C" pararnn_status pararnn_block_selective_scan(const pararnn_block_ssm* q, void* y, const int64_t sy[2], float* h_last,
                                                       float* carry, void* ws, size_t ws_bytes, void* stream) {
  if (!problem_ok(q) || !sy || !plane_ok(q->B, sy[0]) || !plane_ok(q->T, sy[1])) return PARARNN_ERR_INVALID_ARG;
  const bool any = q->B > 0 && q->D > 0;
  if (!ptr_ok(y, dtype_size(q->dtype), any && q->T > 0) || !ptr_ok(h_last, 4, false) || !ptr_ok(carry, 4, false))
    return PARARNN_ERR_INVALID_ARG;
  const Split s = forward_split(q->B, q->T, q->D, q->G);
  if (far(q, sy[1]) || !supported(q, s, waves_of(q->N) * WAVE)) return PARARNN_ERR_UNSUPPORTED;
  const Room r = room(q->B, q->T, q->D, q->N, q->G, false);
  if (!ws_ok(ws, ws_bytes, static_cast<size_t>(r.total()) * sizeof(float))) return PARARNN_ERR_WORKSPACE;
  if (!any) return PARARNN_OK;
  const auto st = static_cast<hipStream_t>(stream);
  SsmArgs p = ssm_args(q, s);
  if (q->T == 0) {
    const int64_t n = q->B * p.seqs.n * q->D * q->N;
    if (!h_last || h_last == q->h0) return PARARNN_OK;
    if (!grid_ok(ceil_div(n, 256), 256)) return PARARNN_ERR_UNSUPPORTED;
    k_copy_states<<<dim3(static_cast<uint32_t>(ceil_div(n, 256))), dim3(256), 0, st>>>(q->h0, h_last, n);
    return launched();
  }
  p.y = y;
  p.sy[0] = sy[0], p.sy[1] = step_of(q, sy[1]);
  p.h_last = h_last, p.carry = carry;
  p.in_place = h_last && h_last == q->h0;
  float* f = static_cast<float*>(ws);
  p.end = f, p.sum = f + r.end;
  p.head = p.in_place ? f + r.end + r.sum : nullptr;
  return q->dtype == PARARNN_BF16 ? by_states<Forward, bf16>(q->N, p, s, st) : by_states<Forward, float>(q->N, p, s, st);
}

extern "C" pararnn_status pararnn_block_selective_scan_vjp(const pararnn_block_ssm* q, const pararnn_block_ssm_grad* grad, void* ws,
                                                           size_t ws_bytes, void* stream) {
  if (!problem_ok(q) || !grad) return PARARNN_ERR_INVALID_ARG;
  const size_t e = dtype_size(q->dtype);
  const bool any = q->B > 0 && q->D > 0, steps = any && q->T > 0;
  if (!ptr_ok(grad->carry, 4, steps) || !ptr_ok(grad->dy, e, steps) || !ptr_ok(grad->d_last, 4, false) ||
      !ptr_ok(grad->d_x, e, steps) || !ptr_ok(grad->d_delta, e, steps) || !ptr_ok(grad->d_z, e, steps && q->z) ||
      !ptr_ok(grad->d_b, e, steps) || !ptr_ok(grad->d_c, e, steps) || !ptr_ok(grad->d_A, 4, false) ||
      !ptr_ok(grad->d_skip, 4, false) || !ptr_ok(grad->d_dt_bias, 4, false) || !ptr_ok(grad->d_h0, 4, false))
    return PARARNN_ERR_INVALID_ARG;
  const int64_t(*s2[4])[2] = {&grad->sdy, &grad->sdx, &grad->sddelta, &grad->sdz};
  for (int k = 0; k < (q->z ? 4 : 3); ++k)
    if (!plane_ok(q->B, (*s2[k])[0]) || !plane_ok(q->T, (*s2[k])[1])) return PARARNN_ERR_INVALID_ARG;
  const int64_t(*s3[2])[3] = {&grad->sdb, &grad->sdc};
  for (const auto* s : s3)
    if (!plane_ok(q->B, (*s)[0]) || !plane_ok(q->T, (*s)[1]) || !plane_ok(q->G, (*s)[2])) return PARARNN_ERR_INVALID_ARG;

  const Split s = gradient_split(q->B, q->T, q->D, q->G);
  const int64_t values = q->B * q->T * q->G * 2 * q->N, cols = q->D * (q->N + 2);
  if (far(q, grad->sdy[1]) || far(q, grad->sdx[1]) || far(q, grad->sddelta[1]) || (q->z && far(q, grad->sdz[1])))
    return PARARNN_ERR_UNSUPPORTED;
  if (!supported(q, s, waves_of(q->N) * WAVE) || !grid_ok(ceil_div(values, 256), 256) || !grid_ok(ceil_div(cols, 64), 256))
    return PARARNN_ERR_UNSUPPORTED;
  const Room r = room(q->B, q->T, q->D, q->N, q->G, true);
  if (!ws_ok(ws, ws_bytes, static_cast<size_t>(r.total()) * sizeof(float))) return PARARNN_ERR_WORKSPACE;
  if (q->D == 0) return PARARNN_OK;
  const auto st = static_cast<hipStream_t>(stream);
  SsmGradArgs g{};
  g.f = ssm_args(q, s);
  SsmArgs& p = g.f;
  float* f = static_cast<float*>(ws);
  p.end = f, p.sum = f + r.end;
  f += r.end + r.sum;
  g.part_bc = f;
  f += r.bc;
  g.part_A = f;
  float* scratch = f + r.part;
  g.carry = grad->carry, g.dy = grad->dy, g.d_last = grad->d_last, g.d_h0 = grad->d_h0;
  g.dx = grad->d_x, g.ddelta = grad->d_delta, g.dz = grad->d_z;
  for (int k = 0; k < 2; ++k)
    g.sdy[k] = grad->sdy[k], g.sdx[k] = grad->sdx[k], g.sddelta[k] = grad->sddelta[k], g.sdz[k] = grad->sdz[k];
  for (int64_t* t : {&g.sdy[1], &g.sdx[1], &g.sddelta[1], &g.sdz[1]}) *t = step_of(q, *t);
  if (steps) {
    const pararnn_status st1 = q->dtype == PARARNN_BF16 ? by_states<Backward, bf16>(q->N, g, s, st)
                                                        : by_states<Backward, float>(q->N, g, s, st);
    if (st1 != PARARNN_OK) return st1;
    SharedArgs a{g.part_bc, q->B, q->T, p.N, p.G, p.ctiles, grad->d_b, grad->d_c, {}, {}};
    for (int k = 0; k < 3; ++k) a.sdb[k] = grad->sdb[k], a.sdc[k] = grad->sdc[k];
    const dim3 grid(static_cast<uint32_t>(ceil_div(values, 256)));
    if (q->dtype == PARARNN_BF16) k_ssm_shared<bf16><<<grid, dim3(256), 0, st>>>(a);
    else k_ssm_shared<float><<<grid, dim3(256), 0, st>>>(a);
  }
  if (grad->d_h0 && any && (q->cu_seqlens || q->T == 0)) {
    const int64_t states = q->D * q->N, n = q->B * p.seqs.n * states;
    if (!grid_ok(ceil_div(n, 256), 256)) return PARARNN_ERR_UNSUPPORTED;
    k_ssm_empty<<<dim3(static_cast<uint32_t>(ceil_div(n, 256))), dim3(256), 0, st>>>(p.seqs, states, n, grad->d_last, grad->d_h0);
  }
  if (grad->d_A || grad->d_skip || grad->d_dt_bias) {
    const ToParams to{q->D, p.N, grad->d_A, grad->d_skip, grad->d_dt_bias};
    if (!colsum(g.part_A, steps ? s.S * q->B : 0, cols, to, scratch, st)) return PARARNN_ERR_UNSUPPORTED;
  }
  return launched();
}
