// lm_scan.hip -- the gated linear recurrence of pararnn_lm.h and its gradients.
//
//   a_t = exp(k sig(r_t)), k = -c softplus(lam);  h_t = a_t h_{t-1} + m_t u_t,  m = sqrt(1 - a^2), u = sig(i) x

#include <algorithm>
#include <type_traits>

#include "lm_common.h"

namespace lm {

constexpr int CT = PARARNN_LM_SCAN_CHUNK;

struct ScanArgs {
  const void *x, *r, *i;
  int64_t sx[2], sr[2], si[2];
  const float* lam;
  const float* h0;
  const int32_t* cu;
  int32_t n;          // sequences of a row (1 without cu)
  float c;
  int64_t B, T, D;
  void* h;
  int64_t sh[2];
  float* h_last;
  float* carry;
};

struct GradArgs {
  ScanArgs f;
  const void* dh;
  const float* d_last;
  void *dx, *dr, *di;
  int64_t sdh[2], sdx[2], sdr[2], sdi[2];
  float* part;        // [B][chunks][D] sums of e sig(r) over a chunk
  float* d_h0;
};

// softplus(x) = max(x, 0) + log1p(e^-|x|); log1p(e) = log(w) e / (w - 1) with w = fl(1 + e), exact in the
// rounding of w (W. Kahan's correction), since small rates (1e-4 and below) set the longest memories
DEV float softplus(float x) {
  const float e = hw_exp2(-kLog2e * fabsf(x));
  const float w = 1.0f + e;
  const float l = w == 1.0f ? e : kLn2 * hw_log2(w) * e * hw_rcp(w - 1.0f);
  return fmaxf(x, 0.0f) + l;
}

// The gates of one element.  For small |log a| q = 1 - a comes first, from the Taylor series of expm1, so that
// a = 1 - q is rounded to nearest and m^2 = 1 - a^2 = q (2 - q) has full relative accuracy (1 - exp() would lose
// it all where a is near 1, which is where these recurrences live); for large |log a| a itself comes first.
// |log a| < |k|: FAR = false is for a k of at most kNear in size, which needs no exponential for a.
struct Gate {
  float a, w, sr, si;   // decay, 1 - a^2, sig(r), sig(i)
};
constexpr float kNear = 0.25f;
template <bool FAR>
DEV Gate gate(float r, float i, float k) {
  Gate g;
  g.sr = sigmoid(r);
  g.si = sigmoid(i);
  const float z = k * g.sr;
  // -expm1(z), |z| <= 1/4: the first term left out is z^6 / 5040 of the sum, 5e-8
  float q = -z * fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.0f / 720.0f, 1.0f / 120.0f), 1.0f / 24.0f), 1.0f / 6.0f),
                              0.5f), 1.0f);
  g.a = 1.0f - q;
  if constexpr (FAR) {
    const float big = hw_exp2(kLog2e * z);
    const bool far = z < -kNear;
    q = far ? 1.0f - big : q;
    g.a = far ? big : g.a;
  }
  g.w = fmaf(q, g.a, q);   // 1 - a^2 = q (1 + a)
  return g;
}
DEV float root(float w) { return __builtin_amdgcn_sqrtf(w); }

// first sequence index j in [0, n) whose steps include t: the number of offsets cu[1 .. n-1] at or below t
DEV int32_t sequence_of(const int32_t* cu, int32_t n, int64_t t) {
  int32_t lo = 0, hi = n - 1;
  while (lo < hi) {
    const int32_t mid = lo + (hi - lo + 1) / 2;
    if (cu[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// ------------------------------------------------------------------------------------------------
// Few steps (kSerial or fewer, one generated token for instance): one channel of one row a thread, all steps
// in order, no shared memory, one launch.
// ------------------------------------------------------------------------------------------------
constexpr int64_t kSerial = 16;   // T = 8, 16, 32: 5.1, 9.9, 16.6 us against the scan's 13.4, 13.8, 14.2 (B = 32, D = 4096, bf16)
template <typename T>
__global__ __launch_bounds__(64) void k_scan_serial(const ScanArgs p, uint32_t ctiles) {
  const int64_t b = blockIdx.x / ctiles, d = static_cast<int64_t>(blockIdx.x - b * ctiles) * 64 + threadIdx.x;
  if (d >= p.D) return;
  const float k = -p.c * softplus(p.lam[d]);
  const T* x = static_cast<const T*>(p.x) + b * p.sx[0] + d;
  const T* r = static_cast<const T*>(p.r) + b * p.sr[0] + d;
  const T* i = static_cast<const T*>(p.i) + b * p.si[0] + d;
  T* out = static_cast<T*>(p.h) + b * p.sh[0] + d;
  const int64_t state = b * p.n * p.D + d;
  int64_t t = 0;
  for (int32_t j = 0; j < p.n; ++j) {
    float h = p.h0 ? p.h0[state + j * p.D] : 0.0f;
    int64_t end = j + 1 < p.n ? p.cu[j + 1] : p.T;
    if (end > p.T) end = p.T;
    for (; t < end; ++t) {
      if (p.carry && t == 0) p.carry[b * p.D + d] = h;
      const Gate g = gate<true>(to_f32(r[t * p.sr[1]]), to_f32(i[t * p.si[1]]), k);
      h = fmaf(g.a, h, root(g.w) * (g.si * to_f32(x[t * p.sx[1]])));
      out[t * p.sh[1]] = from_f32<T>(h);
    }
    if (p.h_last) p.h_last[state + j * p.D] = h;
  }
}

// ------------------------------------------------------------------------------------------------
// The parallel scan.  A tile is one workgroup: CT steps of TW channels of one row.  A lane holds V channels of
// L = 16 / V consecutive steps; the lanes of a wave cover TW channels V times over, as V time slices.  A tile's steps are
// NSEG segments of SL, whatever V is, so that strides and widths change no bit.  Each lane composes its segments' maps
// h -> a h + b; each wave, now a lane a channel, joins its own segments; one wave joins the waves', takes the state
// entering the tile from the tiles before it and gives every wave its entering state, from which each wave finds its
// segments' and the lanes walk their steps.  Inputs are read once.
//
// Between tiles.  Each tile publishes its map for each channel as a 64-bit word; GS tiles of a chain form a group, whose
// last tile joins their maps to the group's and publishes that, then finds the state entering the group -- the nearest
// state among the W groups before it, advanced by the maps of those between -- and replaces the group's map by the state
// leaving it.  Every tile's entering state is its group's, advanced by the joint map of the group's tiles before it.  So a
// state travels 64 tiles in one round trip through memory, and what is composed with what is fixed: every run gives the
// same bits.  a is in [0, 1], so the sign bit of A marks a word as written: zero = nothing yet, (A | sign, B) = a map,
// (~0, h) = a state.  Words are relaxed device-scope atomics and carry their own validity: no fences.
//
// A tile takes its place from a ticket counter, so those it waits for have been started before it.  One counter hands
// out a ticket in 13 ns, which bounded the whole scan; the chains therefore form up to 8 classes with a counter each.  A
// workgroup starts with a class that is no function of its XCD (the block number modulo 8): chains bound to an XCD cost
// 25% at T = 131072, D = 1024.
//
// V = 4, with accesses of 8 or 16 bytes at any alignment of the element; where four does not divide the width the last lane's
// channels overlap the lane's before (two lanes then store the same values).  One element a lane (V = 1) costs 50.8 against
// 46.1 us in the gradient of bf16 B = 2, T = 10301, D = 345 and 11 against 8 us where one tile is all of time; it stays
// for fewer than four channels and for steps too far apart for 32-bit offsets.
//
// Packed sequences: a wave finds its steps' sequences once and keeps them in shared memory (searched for at each boundary
// by its lane: bf16 B = 4, T = 4096, D = 1000, 9 sequences 108 against 93 us in the gradient, 61 against 51 forward).
//
// Bound by memory for float32, by memory and vector instructions about equally for bfloat16 (57% of the issue slots forward,
// 70% in the gradient).  Measured, bf16 (wide: B = 2, T = 4096, D = 4096; long: B = 1, T = 131072, D = 1024): forward 62 and
// 260 us (4.2 TB/s), gradient 109 and 464 to 490 us (4.1 TB/s); a copy runs at 5.1 TB/s.  The forms without packing spill
// nothing (V = 4).  The packed ones spill scalar registers to vector lanes (11 or 12 forward, 29 in the gradient with V = 4, 120
// with V = 1), and the forward bf16 V = 4 one two vector registers: the boundaries' bases stay live through the walks.
//  - 64 steps a tile (4 waves) against 128 (8 waves): gradient 118 against 151 us (wide, when chosen), since its 156 registers leave
//    12 waves on a CU in workgroups of 4 and 8 in workgroups of 8; forward 66 against 72.  32 elements a lane: 66 and 124.
//  - groups against a look-back over the W tiles before: forward 257 against 297 us (long).  Groups of 16: 325.
//  - stores that do not stay in the caches: float32 B = 8, T = 2048, D = 1000 forward 69 against 81 us; wide 62.6 against 64.0.
// ------------------------------------------------------------------------------------------------
constexpr int EPL = 16, NW = CT / EPL, TW = WAVE, NTH = NW * WAVE, W = 8, GS = 8;
static_assert(NW * EPL == CT && NW >= 2, "EPL elements a lane");
constexpr int kStream = 2;   // cache policy of a buffer store: non-temporal
constexpr int SL = 4, NSEG = CT / SL, SW = NSEG / NW;   // steps of a segment, segments of a tile and of a wave
template <int V> struct Shape { static constexpr int L = EPL / V, Q = L / SL; };   // steps and segments of a lane

struct Grid {
  uint64_t* words;      // [chunks][chains][TW]: the tiles' maps
  uint64_t* gwords;     // [chunks / GS][chains][TW]: the groups' maps, then the states leaving them
  uint32_t* tickets;    // a counter for each class of chains, kTicket words apart; null: one chunk, the tile is the block
  int64_t chunks;
  int32_t chains, ctiles, log_classes;   // chains = B ctiles: channel tiles of all rows
};

constexpr int kTicket = 32, kLogClasses = 3;   // 128 bytes: counters share no cache line

struct Aff { float A, B; };
// The map of `later` after `earlier`.  With packed sequences A = NaN is a cut: nothing crosses it, not even a NaN, and the
// product keeps it without a select.  (A = 0 would not do: strong decays have products of zero, which a NaN crosses.)  A map
// whose own decay is NaN has B = NaN too, so that nothing is lost by reading it as a cut.
constexpr float kCut = __builtin_nanf("");
template <bool SEG> DEV float apply(const Aff& f, float h) { return SEG && f.A != f.A ? f.B : fmaf(f.A, h, f.B); }
template <bool SEG> DEV Aff compose(const Aff& later, const Aff& earlier) {
  return {later.A * earlier.A, apply<SEG>(later, earlier.B)};
}

DEV uint64_t ld_word(const uint64_t* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
DEV void st_word(uint64_t* p, uint32_t hi, float lo) {
  __hip_atomic_store(p, (static_cast<uint64_t>(hi) << 32) | __float_as_uint(lo), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
constexpr uint32_t kState = 0xffffffffu, kSign = 0x80000000u;
DEV uint32_t map_bits(float A) { return A != A ? 0xffc00000u : (__float_as_uint(A) | kSign); }

// The stress build (-DPR_LB_STRESS=1) pauses a quarter of the tiles for a bounded, pseudo-random time before they publish a
// word, so that words come in a scrambled order; its results must be the plain library's, bit for bit.
#ifndef PR_LB_STRESS
#define PR_LB_STRESS 0
#endif
DEV void stress_pause(uint32_t pos, int32_t chain, uint32_t site) {
  if constexpr (PR_LB_STRESS) {
    uint32_t h = pos * 0x85EBCA77u ^ static_cast<uint32_t>(chain) * 0xC2B2AE3Du ^ site * 0x27D4EB2Fu ^
                 static_cast<uint32_t>(__builtin_readcyclecounter() >> 8) * 0x9E3779B1u;
    h ^= h >> 15;
    h *= 0x2C1B3C6Du;
    h ^= h >> 12;
    const int n = (h & 3) == 0 ? static_cast<int>((h >> 8) & 31) : 0;   // up to ~100 us
    for (int i = 0; i < n; ++i) __builtin_amdgcn_s_sleep(127);
  }
}

// N words of one channel at `word` - k step for k = 0 .. N-1, those with k >= have not read
template <int N> DEV void ld_words(const uint64_t* word, int64_t step, int have, uint64_t (&w)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) w[k] = k < have ? ld_word(word - k * step) : 0;   // uniform
}
DEV uint32_t hi(uint64_t w) { return static_cast<uint32_t>(w >> 32); }
DEV float lo(uint64_t w) { return __uint_as_float(static_cast<uint32_t>(w)); }
DEV Aff map_of(uint64_t w) { return {__uint_as_float(hi(w) & ~kSign), lo(w)}; }

// The state entering group `j` > 0 of a chain, for this lane's channel: the nearest state among the N groups before it,
// advanced by the maps of the groups between, in order.
template <bool SEG, int N>
DEV float group_state(const Grid& g, uint32_t j, int32_t chain, int lane) {
  const int64_t step = static_cast<int64_t>(g.chains) * TW;
  const uint64_t* word = g.gwords + static_cast<int64_t>(j - 1) * step + static_cast<int64_t>(chain) * TW + lane;
  while (true) {
    uint64_t w[N];
    ld_words(word, step, j < N ? static_cast<int>(j) : N, w);
    int at = -1;          // the nearest state, if every word before it is there
    bool there = true;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if (there && at < 0 && hi(w[k]) == kState) at = k;
      there = there && hi(w[k]) != 0;
    }
    if (at >= 0) {
      float h = 0.0f;
#pragma unroll
      for (int k = N - 1; k >= 0; --k) {
        if (k == at) h = lo(w[k]);
        else if (k < at) h = apply<SEG>(map_of(w[k]), h);
      }
      return h;
    }
    __builtin_amdgcn_s_sleep(1);
  }
}

// The state entering the tile at `pos`, whose own map is f, for this lane's channel; `first` is the one entering the chain.
template <bool SEG> DEV float enter_tile(const Grid& g, uint32_t pos, int32_t chain, int lane, const Aff& f, float first) {
  const int64_t step = static_cast<int64_t>(g.chains) * TW, col = static_cast<int64_t>(chain) * TW + lane;
  const uint32_t j = pos / GS;
  const int i = static_cast<int>(pos % GS);
  const bool more = pos + 1 < g.chunks;
  uint64_t* own = g.words + pos * step + col;
  stress_pause(pos, chain, 0);
  if (more && i + 1 < GS) st_word(own, map_bits(f.A), f.B);
  Aff m{1.0f, 0.0f};   // the group's tiles before this one
  if (i > 0) {
    uint64_t w[GS - 1];
    while (true) {
      ld_words(own - step, step, i, w);
      bool there = true;
#pragma unroll
      for (int k = 0; k < GS - 1; ++k) there = there && (k >= i || hi(w[k]) != 0);
      if (there) break;
      __builtin_amdgcn_s_sleep(1);
    }
#pragma unroll
    for (int k = GS - 2; k >= 0; --k)
      if (k < i) m = k == i - 1 ? map_of(w[k]) : compose<SEG>(map_of(w[k]), m);
  }
  float h;
  if (more && i + 1 == GS) {   // the group's last tile: publishes the group's map, then the state leaving it
    const Aff all = compose<SEG>(f, m);
    uint64_t* group = g.gwords + j * step + col;
    stress_pause(pos, chain, 1);
    if (j > 0) st_word(group, map_bits(all.A), all.B);
    h = j > 0 ? group_state<SEG, W>(g, j, chain, lane) : first;
    stress_pause(pos, chain, 2);
    st_word(group, kState, apply<SEG>(all, h));
  } else {
    h = j > 0 ? group_state<SEG, 4>(g, j, chain, lane) : first;
  }
  return i > 0 ? apply<SEG>(m, h) : h;
}

// what the lanes of a wave wrote to shared memory is there for its other lanes (a wave's accesses are in order; this keeps
// the compiler from moving them)
DEV void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}
// a loaded value is there: what the wave stores from here on cannot overtake the load
DEV void arrived(float& v) { asm volatile("" : "+v"(v) : : "memory"); }
// the maps of N consecutive pieces (a lane's column of them) as one, in scan order
template <bool SEG, bool REV, int N> DEV Aff join(const Aff (*m)[TW], int lane) {
  Aff f = m[REV ? N - 1 : 0][lane];
#pragma unroll
  for (int k = 1; k < N; ++k) f = compose<SEG>(m[REV ? N - 1 - k : k][lane], f);
  return f;
}
// the states entering them, from the one entering the first.  The maps are read again: held since join() they would cost
// the registers of a wave a SIMD.
template <bool SEG, bool REV, int N> DEV void spread(const Aff (*m)[TW], float (*enter)[TW], int lane, float h) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int s = REV ? N - 1 - k : k;
    enter[s][lane] = h;
    if (k + 1 < N) h = apply<SEG>(m[s][lane], h);
  }
}
// the tile's place: its position in its chain.  Chain c is of class c modulo 2^log_classes; a workgroup whose class has no
// ticket left goes on to the next (there are as many workgroups as tiles).
DEV void take_ticket(const Grid& g, uint32_t (&sh)[2], uint32_t& pos, uint32_t& chain) {
  const uint32_t mask = (1u << g.log_classes) - 1, chains = static_cast<uint32_t>(g.chains);
  const auto size = [&](uint32_t n) { return (chains + mask - n) >> g.log_classes; };   // chains of class n
  if (!g.tickets) {
    pos = 0;
    chain = blockIdx.x;
    return;
  }
  if (threadIdx.x == 0) {
    uint32_t n = (blockIdx.x >> 3) & mask, t;
    while ((t = __hip_atomic_fetch_add(g.tickets + n * kTicket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) >=
           size(n) * static_cast<uint32_t>(g.chunks))
      n = (n + 1) & mask;
    sh[0] = t;
    sh[1] = n;
  }
  __syncthreads();
  const uint32_t t = __builtin_amdgcn_readfirstlane(sh[0]), n = __builtin_amdgcn_readfirstlane(sh[1]);
  const uint32_t per = size(n);
  // scalar registers for what every address is made of (else in vector registers: 44 bytes spilled, 92 against 63 us)
  pos = __builtin_amdgcn_readfirstlane(t / per);
  chain = __builtin_amdgcn_readfirstlane(((t - pos * per) << g.log_classes) + n);
}

// where a tile and its lanes are
template <int V>
struct Tile {
  int64_t b, t0, c0, t;   // row, the tile's first step and channel; the lane's first step
  uint32_t pos, chunk;    // place in scan order, chunk
  int32_t chain;
  int seg, ch, lane, wave, slice;   // the lane's first segment and first channel within the tile
  int cols;               // the tile's channels
  bool active, full;      // the lane's channels exist; all the tile's steps do
  int valid;              // steps of the lane below T
  DEV Tile(const Grid& g, const ScanArgs& p, uint32_t (&sh)[2], bool reverse) {
    constexpr int L = Shape<V>::L, Q = Shape<V>::Q;
    lane = threadIdx.x % WAVE;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    uint32_t c;
    take_ticket(g, sh, pos, c);
    chain = static_cast<int32_t>(c);
    chunk = reverse ? static_cast<uint32_t>(g.chunks) - 1 - pos : pos;
    const uint32_t row = static_cast<uint32_t>(chain) / static_cast<uint32_t>(g.ctiles);
    b = row;
    const int32_t column = chain - static_cast<int32_t>(row) * g.ctiles;
    c0 = static_cast<int64_t>(column) * TW;
    cols = p.D - c0 < TW ? static_cast<int>(p.D - c0) : TW;
    if (V > 1) {   // a last tile of fewer than V channels takes V of the one before
      const int rest = static_cast<int>(p.D % TW);
      if (rest > 0 && rest < V) {
        if (column == g.ctiles - 1) c0 -= V, cols += V;
        if (column == g.ctiles - 2) cols -= V;
      }
    }
    t0 = static_cast<int64_t>(chunk) * CT;
    slice = lane / (WAVE / V);
    seg = (wave * V + slice) * Q;
    ch = (lane % (WAVE / V)) * V;
    active = ch < cols;
    if (active && ch > cols - V) ch = cols - V;   // the last V channels, some of them with the lane before: the same values
    t = t0 + seg * SL;
    full = t0 + CT <= p.T;
    valid = L;
    if (!full) {
      const int64_t left = p.T - t;
      valid = static_cast<int>(left < 0 ? 0 : left > L ? L : left);
    }
  }
};

// A plane as a wave sees it: a buffer descriptor that begins at the wave's first step and ends with the row's last step, so
// that no access leaves the row and stores past its end do nothing, without a branch (loads past the end return zero, or a
// step's values where steps overlap); the lane's byte offsets from it are 32 bits.  Lanes without channels are out of range.
// Steps too far apart for that (kFar bytes) go one by one with 64-bit addresses, V = 1 only.
constexpr int64_t kFar = (INT64_C(1) << 31) / EPL;
template <typename T, int V>
struct Plane {
  static constexpr int L = Shape<V>::L;
  char* base;
  int64_t st;      // bytes from step to step
  int32_t steps;   // of the wave, below T
  uint32_t width, off;
  bool far;
  DEV Plane(const void* p, const int64_t (&s)[2], const Tile<V>& tl, const ScanArgs& a) {
    const int64_t t = tl.t0 + tl.wave * (V * L), left = a.T - t;
    st = s[1] * static_cast<int64_t>(sizeof(T));
    base = static_cast<char*>(const_cast<void*>(p)) + (tl.b * s[0] + t * s[1] + tl.c0) * static_cast<int64_t>(sizeof(T));
    steps = static_cast<int32_t>(left < 0 ? 0 : left > V * L ? V * L : left);
    width = static_cast<uint32_t>(tl.cols) * static_cast<uint32_t>(sizeof(T));
    off = static_cast<uint32_t>(tl.slice * L) * static_cast<uint32_t>(st) + static_cast<uint32_t>(tl.ch * sizeof(T));
    if (!tl.active) off = 0x80000000u;   // + 15 steps: still past any end, and no wrap
    far = V == 1 && st > kFar;
  }
  DEV __amdgpu_buffer_rsrc_t all() const {
    const uint32_t bytes = steps > 0 ? static_cast<uint32_t>(steps - 1) * static_cast<uint32_t>(st) + width : 0u;
    return __builtin_amdgcn_make_buffer_rsrc(base, static_cast<short>(0), static_cast<int>(bytes), 0x00020000);
  }
  DEV uint32_t at(int l) const { return off + static_cast<uint32_t>(l) * static_cast<uint32_t>(st); }
  DEV bool has(int l) const { return l < steps && off < width; }   // far, V = 1
  DEV T* element(int l) const { return reinterpret_cast<T*>(base + l * st + off); }
  DEV Vec<T, V> load(int l) const {
    Vec<T, V> r;
    if constexpr (V * sizeof(T) == 2) {
      r.w[0] = __builtin_amdgcn_raw_buffer_load_b16(all(), at(l), 0, 0);
    } else if constexpr (V * sizeof(T) == 4) {
      r.w[0] = __builtin_amdgcn_raw_buffer_load_b32(all(), at(l), 0, 0);
    } else if constexpr (V * sizeof(T) == 8) {
      const auto q = __builtin_amdgcn_raw_buffer_load_b64(all(), at(l), 0, 0);
      r.w[0] = q[0], r.w[1] = q[1];
    } else {
      const auto q = __builtin_amdgcn_raw_buffer_load_b128(all(), at(l), 0, 0);
#pragma unroll
      for (int k = 0; k < 4; ++k) r.w[k] = q[k];
    }
    return r;
  }
  DEV void store(int l, const float (&x)[V]) const {
    const Vec<T, V> r = pack_vec<T, V>(x);
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    if (far) {   // uniform
      if (has(l)) *element(l) = from_f32<T>(x[0]);
    }
    else if constexpr (V * sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(r.w[0]), all(), at(l), 0, kStream);
    else if constexpr (V * sizeof(T) == 4) __builtin_amdgcn_raw_buffer_store_b32(r.w[0], all(), at(l), 0, kStream);
    else if constexpr (V * sizeof(T) == 8) __builtin_amdgcn_raw_buffer_store_b64(u32x2{r.w[0], r.w[1]}, all(), at(l), 0, kStream);
    else __builtin_amdgcn_raw_buffer_store_b128(u32x4{r.w[0], r.w[1], r.w[2], r.w[3]}, all(), at(l), 0, kStream);
  }
};

// one plane's L steps of V channels
template <typename T, int V, int L>
DEV void load_steps(const void* p, const int64_t (&s)[2], const Tile<V>& tl, const ScanArgs& a, Vec<T, V> (&v)[L]) {
  const Plane<T, V> pl(p, s, tl, a);
  if (pl.far) {   // uniform
#pragma unroll
    for (int l = 0; l < L; ++l) {
      v[l].w[0] = 0;
      if (pl.has(l)) {
        const T e = *pl.element(l);
        if constexpr (sizeof(T) == 4) v[l].w[0] = __float_as_uint(e);
        else v[l].w[0] = e.u;
      }
    }
    return;
  }
#pragma unroll
  for (int l = 0; l < L; ++l) v[l] = pl.load(l);
}

// k = -c softplus(lam) of the lane's channels: a lane evaluates one channel of the tile, the others fetch it; `far`: some
// channel of the tile is beyond kNear
template <int V>
DEV bool rates(const ScanArgs& p, const Tile<V>& tl, float (&k)[V]) {
  const int64_t d = tl.c0 + tl.lane < p.D ? tl.c0 + tl.lane : p.D - 1;
  const float own = -p.c * softplus(p.lam[d]);
#pragma unroll
  for (int v = 0; v < V; ++v) k[v] = V == 1 ? own : __shfl(own, tl.ch + v, WAVE);
  return __any(!(own >= -kNear));
}

// Packed sequences: which of the lane's steps begin and which end one (the row's first and last step included), and the
// sequence of each of the wave's steps in `seq`.  The offsets are searched once for the wave's steps together, with scalar
// loads, which do not wait for the planes'.
template <int V>
DEV void boundaries(const ScanArgs& p, const Tile<V>& tl, uint32_t& starts, uint32_t& ends, int32_t (&seq)[EPL]) {
  constexpr int S = V * Shape<V>::L;
  static_assert(S == EPL && S <= 32, "the steps of a wave are bits of a word");
  const int64_t t = tl.t0 + tl.wave * S;
  starts = ends = 0;
  if (t >= p.T) return;
  const int left = static_cast<int>(p.T - t < S ? p.T - t : S);
  int32_t j = sequence_of(p.cu, p.n, t), mine = j;   // mine: of step number `lane`
  if (t == 0 || (j > 0 && p.cu[j] == t)) starts = 1;
  for (++j; j < p.n; ++j) {   // the sequences that begin after step t
    const int64_t at = p.cu[j] - t;
    if (at > left || at < 1) break;   // at < 1: offsets out of order
    ends |= 1u << (at - 1);
    if (at < left) starts |= 1u << at;
    if (tl.lane >= at) mine = j;
  }
  if (tl.lane < S) seq[tl.lane] = mine;
  wave_sync();
  if (t + left == p.T) ends |= 1u << (left - 1);
  starts = starts >> (tl.slice * Shape<V>::L) & (~0u >> (32 - Shape<V>::L));
  ends = ends >> (tl.slice * Shape<V>::L) & (~0u >> (32 - Shape<V>::L));
}

template <typename T, int V, bool SEG>
__global__ __launch_bounds__(NTH) __attribute__((amdgpu_waves_per_eu(5))) void k_scan(const ScanArgs p, const Grid g) {
  constexpr int L = Shape<V>::L, Q = Shape<V>::Q;
  __shared__ uint32_t sh_ticket[2];
  __shared__ int32_t sh_seq[SEG ? NW : 1][EPL];
  __shared__ Aff sh_map[NSEG][TW], sh_wave[NW][TW];
  __shared__ float sh_enter[NSEG][TW], sh_in[NW][TW];
  const Tile<V> tl(g, p, sh_ticket, false);

  float a[L][V], b[L][V];
  uint32_t starts = 0, ends = 0;
  {
    Vec<T, V> x[L], r[L], i[L];
    load_steps(p.r, p.sr, tl, p, r);
    load_steps(p.i, p.si, tl, p, i);
    load_steps(p.x, p.sx, tl, p, x);
    float k[V];
    const auto gates = [&](auto far) {
#pragma unroll
      for (int l = 0; l < L; ++l)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const Gate q = gate<decltype(far)::value>(r[l].get(v), i[l].get(v), k[v]);
          a[l][v] = q.a;
          b[l][v] = root(q.w) * (q.si * x[l].get(v));
        }
    };
    if (rates(p, tl, k)) gates(std::true_type{});
    else gates(std::false_type{});
  }
  if (SEG) boundaries(p, tl, starts, ends, sh_seq[tl.wave]);
  if (!tl.full) {   // steps past the end change nothing that is used: no step before them depends on their b
#pragma unroll
    for (int l = 0; l < L; ++l)
#pragma unroll
      for (int v = 0; v < V; ++v) a[l][v] = l < tl.valid ? a[l][v] : 1.0f;
  }
  if (SEG && starts) {
#pragma unroll
    for (int l = 0; l < L; ++l)
      if (starts >> l & 1) {
        const int64_t state = (tl.b * p.n + sh_seq[tl.wave][tl.slice * L + l]) * p.D + tl.c0 + (tl.active ? tl.ch : 0);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (p.h0) b[l][v] = fmaf(a[l][v], p.h0[state + v], b[l][v]);
          a[l][v] = kCut;
        }
      }
  }
#pragma unroll
  for (int s = 0; s < Q; ++s)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      Aff f{a[s * SL][v], b[s * SL][v]};
#pragma unroll
      for (int l = s * SL + 1; l < (s + 1) * SL; ++l) f = compose<SEG>(Aff{a[l][v], b[l][v]}, f);
      sh_map[tl.seg + s][tl.ch + v] = f;
    }
  wave_sync();
  sh_wave[tl.wave][tl.lane] = join<SEG, false, SW>(sh_map + tl.wave * SW, tl.lane);
  __syncthreads();
  if (tl.wave == 0) {
    const int64_t d = tl.c0 + tl.lane;
    float h = 0.0f;
    if (tl.lane < tl.cols) {
      // h0 before anything is published: h_last may be the same array, and a tile that waits for this one's map may write it
      float begin = 0.0f;      // the state of a sequence that begins with the tile
      bool begins = false;
      if (SEG) {
        const int32_t j = sh_seq[0][0];
        begins = tl.t0 == 0 || (j > 0 && p.cu[j] == tl.t0);
        if (begins && p.h0 && p.carry) begin = p.h0[(tl.b * p.n + j) * p.D + d];
      } else if (tl.pos < GS && p.h0) {
        begin = p.h0[tl.b * p.D + d];
      }
      arrived(begin);
      h = enter_tile<SEG>(g, tl.pos, tl.chain, tl.lane, join<SEG, false, NW>(sh_wave, tl.lane), SEG ? 0.0f : begin);
      if (p.carry) p.carry[(tl.b * g.chunks + tl.chunk) * p.D + d] = SEG && begins ? begin : h;
    }
    spread<SEG, false, NW>(sh_wave, sh_in, tl.lane, h);
  }
  __syncthreads();
  spread<SEG, false, SW>(sh_map + tl.wave * SW, sh_enter + tl.wave * SW, tl.lane, sh_in[tl.wave][tl.lane]);
  wave_sync();
  float h[V];
  const Plane<T, V> out(p.h, p.sh, tl, p);
  // the step (of the lane) that ends the row
  const int last = !SEG && tl.chunk + 1 == g.chunks && p.h_last ? static_cast<int>(p.T - 1 - tl.t) : -1;
#pragma unroll
  for (int l = 0; l < L; ++l) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (l % SL == 0) h[v] = sh_enter[tl.seg + l / SL][tl.ch + v];
      h[v] = apply<SEG>(Aff{a[l][v], b[l][v]}, h[v]);
    }
    out.store(l, h);
    if ((SEG ? (ends >> l & 1) && p.h_last : l == last) && tl.active) {
      const int32_t j = SEG ? sh_seq[tl.wave][tl.slice * L + l] : 0;
#pragma unroll
      for (int v = 0; v < V; ++v) p.h_last[(tl.b * p.n + j) * p.D + tl.c0 + tl.ch + v] = h[v];
    }
  }
}

// ------------------------------------------------------------------------------------------------
// The gradients: the same tiles from the last chunk to the first.  A lane holds its steps' gates; the state entering
// the tile (carry) gives h_{t-1} by the forward walk, and the adjoint mu_t = a_t l_t, l_t = dh_t + mu_{t+1}, is the same
// kind of scan (map mu -> a (dh + mu)) run backwards, whose maps share the products of a with the forward one.
//
// The gradients of the gates need both s = sig(v) and 1 - s, each with its own relative accuracy: of an open gate (v > 0) 1 - s
// from s has lost it (1% off at v = 12, zero from 18 on).  e^-v s has it, and then 1 - (1 - s) gives s.  A lane keeps the smaller
// of the two, its sign bit set where it is 1 - s: as many registers as s alone.  The instructions that this takes (12 to 14 an
// element) cost 3% of a bfloat16 training pass (B = 2, T = 4096, D = 4096: 167 -> 172 us) and 0.5% of a packed float32 one
// (191 -> 192).
// ------------------------------------------------------------------------------------------------
DEV float smaller(float v, float s) {   // e^-v s of a shut gate may be infinity times 0: fminf passes a NaN over
  return __builtin_copysignf(fminf(hw_exp2(-kLog2e * v) * s, s), -v);
}
struct Pair { float s, rest; };   // sig(v), 1 - sig(v)
DEV Pair both(float x) {
  const float y = fabsf(x), z = 1.0f - y;
  return __float_as_uint(x) >> 31 ? Pair{z, y} : Pair{y, z};
}
template <typename T, int V, bool SEG>
__global__ __launch_bounds__(NTH) __attribute__((amdgpu_waves_per_eu(3))) void k_scan_grad(const GradArgs q, const Grid g) {
  constexpr int L = Shape<V>::L, Q = Shape<V>::Q;
  const ScanArgs& p = q.f;
  __shared__ uint32_t sh_ticket[2];
  __shared__ int32_t sh_seq[SEG ? NW : 1][EPL];
  __shared__ Aff sh_fwd[NSEG][TW], sh_rev[NSEG][TW], sh_wfwd[NW][TW], sh_wrev[NW][TW];
  __shared__ float sh_h[NSEG][TW], sh_mu[NSEG][TW], sh_wh[NW][TW], sh_wmu[NW][TW];
  const Tile<V> tl(g, p, sh_ticket, true);

  // kept of each element: a, m, the input m u, sig(r) and sig(i) or their complements; dh in its storage type
  Vec<T, V> dh[L];
  float a[L][V], in[L][V], m[L][V], sr[L][V], si[L][V], k[V];
  uint32_t starts = 0, ends = 0;
  {
    Vec<T, V> x[L], r[L], i[L];
    load_steps(p.r, p.sr, tl, p, r);
    load_steps(p.i, p.si, tl, p, i);
    load_steps(p.x, p.sx, tl, p, x);
    load_steps(q.dh, q.sdh, tl, p, dh);
    if (SEG) boundaries(p, tl, starts, ends, sh_seq[tl.wave]);
    const auto gates = [&](auto far) {
#pragma unroll
      for (int l = 0; l < L; ++l)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const Gate t = gate<decltype(far)::value>(r[l].get(v), i[l].get(v), k[v]);
          a[l][v] = t.a;
          sr[l][v] = smaller(r[l].get(v), t.sr);
          si[l][v] = smaller(i[l].get(v), t.si);
          m[l][v] = root(t.w);
          in[l][v] = m[l][v] * (t.si * x[l].get(v));
        }
    };
    if (rates(p, tl, k)) gates(std::true_type{});
    else gates(std::false_type{});
  }
  if (!tl.full) {   // steps past the end change nothing and add nothing, whatever a plane of overlapping steps has there
#pragma unroll
    for (int l = 0; l < L; ++l) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        a[l][v] = l < tl.valid ? a[l][v] : 1.0f;
        in[l][v] = l < tl.valid ? in[l][v] : 0.0f;
        sr[l][v] = l < tl.valid ? sr[l][v] : 0.0f;
      }
#pragma unroll
      for (int n = 0; n < Vec<T, V>::N; ++n) dh[l].w[n] = l < tl.valid ? dh[l].w[n] : 0u;
    }
  }
  // what enters at a boundary: h0 at a sequence's first step, d_last at its last
  const int64_t dc = tl.c0 + (tl.active ? tl.ch : 0);
  const auto at = [&](const float* base, int l, int v) {
    return base ? base[(tl.b * p.n + sh_seq[tl.wave][tl.slice * L + l]) * p.D + dc + v] : 0.0f;
  };
#pragma unroll
  for (int s = 0; s < Q; ++s)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      Aff f{1.0f, 0.0f}, r{1.0f, 0.0f};
#pragma unroll
      for (int l = s * SL; l < (s + 1) * SL; ++l) {
        Aff e{a[l][v], in[l][v]};
        if (SEG && starts >> l & 1) e = Aff{kCut, fmaf(e.A, at(p.h0, l, v), e.B)};
        f = l % SL ? compose<SEG>(e, f) : e;
      }
#pragma unroll
      for (int l = (s + 1) * SL - 1; l >= s * SL; --l) {
        const bool first = l % SL == SL - 1;   // in scan order
        float mu = r.B, A = first ? a[l][v] : a[l][v] * r.A;
        if (SEG && ends >> l & 1) {
          mu = at(q.d_last, l, v);
          A = kCut;
        }
        r = Aff{A, a[l][v] * (first && !SEG ? dh[l].get(v) : dh[l].get(v) + mu)};
      }
      sh_fwd[tl.seg + s][tl.ch + v] = f;
      sh_rev[tl.seg + s][tl.ch + v] = r;
    }
  wave_sync();
  sh_wfwd[tl.wave][tl.lane] = join<SEG, false, SW>(sh_fwd + tl.wave * SW, tl.lane);
  sh_wrev[tl.wave][tl.lane] = join<SEG, true, SW>(sh_rev + tl.wave * SW, tl.lane);
  __syncthreads();
  const int64_t dl = tl.c0 + tl.lane;
  if (tl.wave == 0) {
    float mu = 0.0f;
    if (tl.lane < tl.cols) {
      if (!SEG && tl.pos < GS) mu = q.d_last ? q.d_last[tl.b * p.D + dl] : 0.0f;
      mu = enter_tile<SEG>(g, tl.pos, tl.chain, tl.lane, join<SEG, true, NW>(sh_wrev, tl.lane), mu);
    }
    spread<SEG, true, NW>(sh_wrev, sh_wmu, tl.lane, mu);
  }
  if (tl.wave == 1)
    spread<SEG, false, NW>(sh_wfwd, sh_wh, tl.lane, tl.lane < tl.cols ? p.carry[(tl.b * g.chunks + tl.chunk) * p.D + dl] : 0.0f);
  __syncthreads();
  spread<SEG, false, SW>(sh_fwd + tl.wave * SW, sh_h + tl.wave * SW, tl.lane, sh_wh[tl.wave][tl.lane]);
  spread<SEG, true, SW>(sh_rev + tl.wave * SW, sh_mu + tl.wave * SW, tl.lane, sh_wmu[tl.wave][tl.lane]);
  wave_sync();
  float sum[Q][V];
#pragma unroll
  for (int s = 0; s < Q; ++s)
#pragma unroll
    for (int v = 0; v < V; ++v) sum[s][v] = 0.0f;
  {
    float mu[V], hq[L][V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float h = 0.0f;
#pragma unroll
      for (int l = 0; l < L; ++l) {
        if (l % SL == 0) h = sh_h[tl.seg + l / SL][tl.ch + v];
        if (SEG && starts >> l & 1) h = at(p.h0, l, v);
        // hq = e / (l a sig(r)) = h_{t-1} - u a / m, where u = in / m
        const float im = m[l][v] > 0.0f ? hw_rcp(m[l][v]) : 0.0f;
        hq[l][v] = fmaf(-in[l][v] * im, a[l][v] * im, h);
        h = fmaf(a[l][v], h, in[l][v]);
      }
    }
    const Plane<T, V> dx(q.dx, q.sdx, tl, p), dr(q.dr, q.sdr, tl, p), di(q.di, q.sdi, tl, p);
    const bool first = !SEG && tl.t == 0 && q.d_h0 && tl.active;
#pragma unroll
    for (int l = L - 1; l >= 0; --l) {
      float ox[V], og[V], oi[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (l % SL == SL - 1) mu[v] = sh_mu[tl.seg + l / SL][tl.ch + v];
        if (SEG && ends >> l & 1) mu[v] = at(q.d_last, l, v);
        const float lam = dh[l].get(v) + mu[v];
        mu[v] = a[l][v] * lam;
        const Pair gr = both(sr[l][v]), gi = both(si[l][v]);
        const float e = mu[v] * hq[l][v] * gr.s;
        sum[l / SL][v] += e;
        og[v] = e * k[v] * gr.rest;
        oi[v] = lam * in[l][v] * gi.rest;
        ox[v] = lam * m[l][v] * gi.s;
      }
      dx.store(l, ox);
      dr.store(l, og);
      di.store(l, oi);
      if (SEG ? (starts >> l & 1) && q.d_h0 && tl.active : l == 0 && first) {
        const int32_t j = SEG ? sh_seq[tl.wave][tl.slice * L + l] : 0;
#pragma unroll
        for (int v = 0; v < V; ++v) q.d_h0[(tl.b * p.n + j) * p.D + dc + v] = mu[v];
      }
    }
  }
  if (!q.part) return;
  // the segments' sums in order, a wave's first (its rows of sh_h are free again), then the waves'
  wave_sync();
#pragma unroll
  for (int s = 0; s < Q; ++s)
#pragma unroll
    for (int v = 0; v < V; ++v) sh_h[tl.seg + s][tl.ch + v] = sum[s][v];
  wave_sync();
  float s = 0.0f;
#pragma unroll
  for (int n = 0; n < SW; ++n) s += sh_h[tl.wave * SW + n][tl.lane];
  sh_wh[tl.wave][tl.lane] = s;
  __syncthreads();
  if (tl.wave == 0 && tl.lane < tl.cols) {
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) s += sh_wh[w][tl.lane];
    q.part[(tl.b * g.chunks + tl.chunk) * p.D + dl] = s;
  }
}

// before a scan: the words and the ticket are cleared, and sequences without a step pass their state on (from `in`, zeros
// when null, to `out`)
__global__ __launch_bounds__(256) void k_scan_prepare(uint4* clear, int64_t n16, const int32_t* cu, int32_t n, int64_t B,
                                                      int64_t T, int64_t D, const float* in, float* out) {
  const int64_t stride = static_cast<int64_t>(gridDim.x) * 256, first = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  for (int64_t k = first; k < n16; k += stride) clear[k] = make_uint4(0u, 0u, 0u, 0u);
  if (!out) return;
  for (int64_t k = first; k < B * n * D; k += stride) {
    const int32_t j = static_cast<int32_t>(k / D % n);
    int64_t t0 = j > 0 ? cu[j] : 0, t1 = j + 1 < n ? cu[j + 1] : T;
    t0 = t0 < 0 ? 0 : t0 > T ? T : t0;
    t1 = t1 < 0 ? 0 : t1 > T ? T : t1;
    if (t0 >= t1) out[k] = in ? in[k] : 0.0f;
  }
}

// d_lam = -c sig(lam) times the sum of the chunks' parts: a workgroup sums kDlam channels, every quarter of a wave every 64th
// row, eight loads at a time, and the quarters' sums are added in order (2048 rows of 1024 channels: 9 us, and 14 with 64
// channels a workgroup)
constexpr int kDlam = 16;
__global__ __launch_bounds__(1024) void k_scan_dlam(const float* part, int64_t rows, int64_t D, const float* lam, float c,
                                                    float* d_lam) {
  constexpr int G = 1024 / kDlam;
  __shared__ float sh[G][kDlam];
  const int ch = threadIdx.x % kDlam, group = threadIdx.x / kDlam;
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * kDlam; first < D; first += static_cast<int64_t>(gridDim.x) * kDlam) {
    const int64_t d = first + ch, dc = d < D ? d : D - 1;
    float s = 0.0f;
    for (int64_t n = group; n < rows; n += G * 8) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = n + u * G < rows ? part[(n + u * G) * D + dc] : 0.0f;
#pragma unroll
      for (int u = 0; u < 8; ++u) s += v[u];
    }
    __syncthreads();   // the channels before have been read
    sh[group][ch] = s;
    __syncthreads();
    if (group == 0 && d < D) {
      s = 0.0f;
#pragma unroll
      for (int k = 0; k < G; ++k) s += sh[k][ch];
      d_lam[d] = -c * sigmoid(lam[d]) * s;
    }
  }
}

// ---------------- host ----------------
static pararnn_status check_scan(const pararnn_lm_scan* p) {
  if (!p || !dtype_ok(p->dtype)) return PARARNN_ERR_INVALID_ARG;
  if (!(p->c > 0.0f) || !std::isfinite(p->c)) return PARARNN_ERR_INVALID_ARG;
  if (!sizes_fit(p->B, p->T, p->D)) return PARARNN_ERR_INVALID_ARG;
  if (p->cu_seqlens && (!aligned(p->cu_seqlens, 4) || p->n_seqs < 1 || p->n_seqs > INT32_MAX - 1 || p->T > INT32_MAX))
    return PARARNN_ERR_INVALID_ARG;
  if (p->cu_seqlens && !sizes_fit(p->B, p->n_seqs, p->D)) return PARARNN_ERR_INVALID_ARG;
  if (!ptr_ok(p->h0, 4, false)) return PARARNN_ERR_INVALID_ARG;
  if (p->D == 0) return PARARNN_OK;
  if (!ptr_ok(p->lam, 4)) return PARARNN_ERR_INVALID_ARG;
  if (p->B == 0) return PARARNN_OK;
  const size_t es = dtype_size(p->dtype);
  if (p->T > 0 && (!ptr_ok(p->x, es) || !ptr_ok(p->r, es) || !ptr_ok(p->i, es))) return PARARNN_ERR_INVALID_ARG;
  const int64_t* s[3] = {p->sx, p->sr, p->si};
  for (const int64_t* q : s)
    if (!plane_ok(p->B, q[0]) || !plane_ok(p->T, q[1])) return PARARNN_ERR_INVALID_ARG;
  return PARARNN_OK;
}

// the strides of a plane of T steps of D channels; that of a single step means nothing, and is made one that a Plane can use
static void strides(int64_t (&to)[2], const int64_t (&from)[2], int64_t T, int64_t D) {
  to[0] = from[0];
  to[1] = T > 1 ? from[1] : D;
}
static ScanArgs scan_args(const pararnn_lm_scan* p) {
  ScanArgs a{};
  a.x = p->x; a.r = p->r; a.i = p->i;
  strides(a.sx, p->sx, p->T, p->D);
  strides(a.sr, p->sr, p->T, p->D);
  strides(a.si, p->si, p->T, p->D);
  a.lam = p->lam; a.h0 = p->h0; a.cu = p->cu_seqlens;
  a.n = p->cu_seqlens ? static_cast<int32_t>(p->n_seqs) : 1;
  a.c = p->c; a.B = p->B; a.T = p->T; a.D = p->D;
  return a;
}

// the workspace: [tickets][words][group words][parts]
struct Layout {
  int64_t chunks, ctiles, tiles, tickets, words, gwords, parts, total;   // the last five in bytes
};
static bool layout(int64_t B, int64_t T, int64_t D, Layout& o) {
  if (!sizes_fit(B, T, D) || D > INT64_MAX - TW || !sizes_fit(B, D + TW, CT)) return false;
  o.chunks = B > 0 && D > 0 ? ceil_div(T, CT) : 0;   // nothing to solve: T alone may be of any size
  o.ctiles = ceil_div(D, TW);
  o.tiles = B * o.ctiles * o.chunks;
  o.words = o.chunks > 1 ? o.tiles * TW * 8 : 0;
  o.tickets = o.chunks > 1 ? (kTicket * 4 << kLogClasses) : 0;
  o.gwords = B * o.ctiles * (o.chunks / GS) * TW * 8;
  o.parts = B * o.chunks * D * 4;
  o.total = 256 + o.tickets + o.words + o.gwords + o.parts;
  return true;
}

// a wave's steps of a plane lie within 32-bit byte offsets
static bool near(const int64_t (&s)[2], size_t es) { return s[1] <= kFar / static_cast<int64_t>(es); }

template <class F>
static void pick(int dtype, bool vec, bool seg, F f) {
  const auto types = [&](auto t) {
    using T = decltype(t);
    if (vec) seg ? f(T{}, std::integral_constant<int, 4>{}, std::true_type{}) : f(T{}, std::integral_constant<int, 4>{}, std::false_type{});
    else seg ? f(T{}, std::integral_constant<int, 1>{}, std::true_type{}) : f(T{}, std::integral_constant<int, 1>{}, std::false_type{});
  };
  if (dtype == PARARNN_BF16) types(bf16{});
  else types(float{});
}

// clears the words where there is more than one chunk, and hands states through empty sequences
static void prepare(const Layout& l, void* ws, const ScanArgs& a, const float* in, float* out, hipStream_t st) {
  const bool empty = out && (a.cu || a.T == 0);
  const int64_t n16 = (l.tickets + l.words + l.gwords) / 16;
  if (!n16 && !empty) return;
  const int64_t work = empty ? std::max(n16, a.B * a.n * a.D) : n16;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(ceil_div(work, 256), 2048));
  k_scan_prepare<<<grid, 256, 0, st>>>(static_cast<uint4*>(ws), n16, a.cu, a.n, a.B, a.T, a.D, in, empty ? out : nullptr);
}
static Grid grid_of(const Layout& l, void* ws, int64_t B) {
  int32_t log = 0;
  while (log < kLogClasses && B * l.ctiles >> (log + 1)) ++log;
  char* w = static_cast<char*>(ws);
  return Grid{reinterpret_cast<uint64_t*>(w + l.tickets), reinterpret_cast<uint64_t*>(w + l.tickets + l.words), l.chunks > 1 ? reinterpret_cast<uint32_t*>(w) : nullptr, l.chunks,
              static_cast<int32_t>(B * l.ctiles), static_cast<int32_t>(l.ctiles), log};
}

}  // namespace lm

using namespace lm;

extern "C" int64_t pararnn_lm_scan_chunks(int64_t T) { return T <= 0 ? 0 : ceil_div(T, CT); }

extern "C" size_t pararnn_lm_scan_workspace_bytes(int64_t B, int64_t T, int64_t D) {
  Layout l;
  return layout(B, T, D, l) ? static_cast<size_t>(l.total) : 0;
}

extern "C" pararnn_status pararnn_lm_gated_scan(const pararnn_lm_scan* prob, void* h, const int64_t sh[2], float* h_last,
                                                float* carry, void* ws, size_t ws_bytes, void* stream) {
  if (const pararnn_status st = check_scan(prob)) return st;
  if (!sh || !ptr_ok(h_last, 4, false) || !ptr_ok(carry, 4, false)) return PARARNN_ERR_INVALID_ARG;
  if (prob->B == 0 || prob->D == 0) return PARARNN_OK;
  const size_t es = dtype_size(prob->dtype);
  if (prob->T > 0 && (!ptr_ok(h, es) || !plane_ok(prob->B, sh[0]) || !plane_ok(prob->T, sh[1])))
    return PARARNN_ERR_INVALID_ARG;
  Layout l;
  if (!layout(prob->B, prob->T, prob->D, l)) return PARARNN_ERR_INVALID_ARG;
  if (!grid_ok(l.tiles, NTH) || !grid_ok(prob->B * l.ctiles, NTH)) return PARARNN_ERR_UNSUPPORTED;
  if (!ptr_ok(ws, 256) || ws_bytes < static_cast<size_t>(l.total)) return PARARNN_ERR_WORKSPACE;
  ScanArgs a = scan_args(prob);
  a.h = h; a.h_last = h_last; a.carry = carry;
  a.sh[0] = sh[0]; a.sh[1] = a.T > 1 ? sh[1] : a.D;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (a.T <= kSerial) {
    const uint32_t ctiles = static_cast<uint32_t>(l.ctiles), grid = static_cast<uint32_t>(a.B) * ctiles;
    if (prob->dtype == PARARNN_BF16) k_scan_serial<bf16><<<grid, 64, 0, st>>>(a, ctiles);
    else k_scan_serial<float><<<grid, 64, 0, st>>>(a, ctiles);
    return launched();
  }
  prepare(l, ws, a, a.h0, a.h_last, st);
  const bool vec = a.D >= 4 && near(a.sx, es) && near(a.sr, es) && near(a.si, es) && near(a.sh, es);
  const Grid g = grid_of(l, ws, a.B);
  pick(prob->dtype, vec, a.cu != nullptr, [&](auto t, auto v, auto seg) {
    k_scan<decltype(t), decltype(v)::value, decltype(seg)::value><<<static_cast<unsigned>(l.tiles), NTH, 0, st>>>(a, g);
  });
  return launched();
}

extern "C" pararnn_status pararnn_lm_gated_scan_vjp(const pararnn_lm_scan* prob, const pararnn_lm_scan_grad* gr, void* ws,
                                                    size_t ws_bytes, void* stream) {
  if (const pararnn_status st = check_scan(prob)) return st;
  if (!gr || !ptr_ok(gr->d_last, 4, false) || !ptr_ok(gr->d_lam, 4, false) || !ptr_ok(gr->d_h0, 4, false))
    return PARARNN_ERR_INVALID_ARG;
  if (prob->D == 0) return PARARNN_OK;
  const size_t es = dtype_size(prob->dtype);
  if (prob->B > 0 && prob->T > 0) {
    if (!ptr_ok(gr->carry, 4) || !ptr_ok(gr->dh, es) || !ptr_ok(gr->d_x, es) || !ptr_ok(gr->d_r, es) ||
        !ptr_ok(gr->d_i, es))
      return PARARNN_ERR_INVALID_ARG;
    const int64_t* s[4] = {gr->sdh, gr->sdx, gr->sdr, gr->sdi};
    for (const int64_t* q : s)
      if (!plane_ok(prob->B, q[0]) || !plane_ok(prob->T, q[1])) return PARARNN_ERR_INVALID_ARG;
  }
  Layout l;
  if (!layout(prob->B, prob->T, prob->D, l)) return PARARNN_ERR_INVALID_ARG;
  if (!grid_ok(l.tiles, NTH) || !grid_ok(prob->B * l.ctiles, NTH)) return PARARNN_ERR_UNSUPPORTED;
  if (!ptr_ok(ws, 256) || ws_bytes < static_cast<size_t>(l.total)) return PARARNN_ERR_WORKSPACE;
  GradArgs q{};
  q.f = scan_args(prob);
  q.f.carry = const_cast<float*>(gr->carry);
  q.dh = gr->dh; q.d_last = gr->d_last; q.dx = gr->d_x; q.dr = gr->d_r; q.di = gr->d_i; q.d_h0 = gr->d_h0;
  strides(q.sdh, gr->sdh, prob->T, prob->D);
  strides(q.sdx, gr->sdx, prob->T, prob->D);
  strides(q.sdr, gr->sdr, prob->T, prob->D);
  strides(q.sdi, gr->sdi, prob->T, prob->D);
  q.part = gr->d_lam ? reinterpret_cast<float*>(static_cast<char*>(ws) + l.tickets + l.words + l.gwords) : nullptr;
  const ScanArgs& a = q.f;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (a.B > 0) prepare(l, ws, a, q.d_last, q.d_h0, st);
  if (l.tiles > 0) {
    const bool vec = a.D >= 4 && near(a.sx, es) && near(a.sr, es) && near(a.si, es) && near(q.sdh, es) && near(q.sdx, es) &&
                     near(q.sdr, es) && near(q.sdi, es);
    const Grid g = grid_of(l, ws, a.B);
    pick(prob->dtype, vec, a.cu != nullptr, [&](auto t, auto v, auto seg) {
      k_scan_grad<decltype(t), decltype(v)::value, decltype(seg)::value><<<static_cast<unsigned>(l.tiles), NTH, 0, st>>>(q, g);
    });
  }
  if (gr->d_lam)
    k_scan_dlam<<<static_cast<unsigned>(std::min<int64_t>(ceil_div(a.D, kDlam), 1 << 16)), 1024, 0, st>>>(q.part, a.B * l.chunks, a.D, a.lam, a.c, gr->d_lam);
  return launched();
}

extern "C" int pararnn_lm_abi_version(void) { return PARARNN_LM_ABI_VERSION; }
