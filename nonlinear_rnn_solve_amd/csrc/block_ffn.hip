// block_ffn.hip -- the gated feed-forward product of pararnn_block.h and its gradients.
//
//   g = x Wg^T, u = x Wu^T, h = act(g) u;   dg = dh u act'(g), du = dh act(g);
//   d_x = dg Wg + du Wu,  d_Wg = dg^T x,  d_Wu = du^T x

#include <algorithm>
#include <type_traits>

#include "block_common.h"

namespace lm {

// ------------------------------------------------------------------------------------------------
// One matrix product serves all of them: C[m][n] = sum_k A[m][k] B[n][k], both operands dense along k.  The forward pass has
// them so as they are; for the gradients the pass that forms dg and du writes them transposed too, and x and the weights are
// transposed into the workspace, with k padded by zeros.
// ------------------------------------------------------------------------------------------------
using v16f = float __attribute__((ext_vector_type(16)));
using v4f = float __attribute__((ext_vector_type(4)));
using v8b = __bf16 __attribute__((ext_vector_type(8)));
using v4u = uint32_t __attribute__((ext_vector_type(4)));

constexpr int kKBytes = 128;    // of k in a tile: 64 bfloat16 or 32 float32
constexpr int kPad = 64;        // k of a transposed operand is a multiple of it
constexpr int planes_of(size_t e) { return e == 2 ? 2 : 1; }    // numbers that make one of dg and du in the gradient's products

// activations and their slopes
template <int ACT> DEV float act(float g) {
  if constexpr (ACT == PARARNN_BLOCK_SILU) return g * sigmoid(g);
  // g Phi(g) ~ g sig(2 sqrt(2 / pi) (g + 0.044715 g^3))
  return g * sigmoid(1.5957691216057308f * fmaf(0.044715f * g, g * g, g));
}
template <int ACT> DEV float slope(float g) {
  if constexpr (ACT == PARARNN_BLOCK_SILU) {
    const float s = sigmoid(g);
    return silu_slope(g, s);
  }
  // beyond 16 the sigmoid is 0 or 1 and the slope too, where g^3 could still pass float32's range (and 0 times infinity follow)
  g = fabsf(g) > 16.0f ? copysignf(16.0f, g) : g;
  const float s = sigmoid(1.5957691216057308f * fmaf(0.044715f * g, g * g, g));
  return s * fmaf(g * (1.0f - s), 1.5957691216057308f * fmaf(3 * 0.044715f * g, g, 1.0f), 1.0f);
}

struct GemmArgs {
  const void *a, *b0, *b1;      // b1: the second weight (forward)
  int64_t sa, sb0, sb1;
  int64_t M, N, K;              // N: of one weight
  int64_t Kb;                   // of B, which is walked anew for each Kb of A's K (K but for two planes, see below)
  void *c0, *c1;                // rows from `split` on go to c1
  int64_t sc0, sc1, split;
  float* pre;
  float* sums;                  // of parts of k
  int64_t per_part;
  int32_t parts;
};

// 16 bytes of a row from element k on, zeros past its n elements
template <typename T> DEV v4u load16(const T* row, int64_t k, int64_t n) {
  constexpr int V = 16 / sizeof(T);
  const Vec<T, V> v = load_row<T, V>(row + k, n - k, T{});
  return v4u{v.w[0], v.w[1], v.w[2], v.w[3]};
}
DEV int64_t at_most(int64_t i, int64_t last) { return i < last ? i : last; }

// the products of 16 bytes of k of each lane: 32 rows by 32 columns, two lanes a row (their halves of k)
template <typename T> DEV void mma(const v4u& a, const v4u& b, v16f& c) {
  if constexpr (sizeof(T) == 2) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0, 0);
  } else {
    const v4f x = __builtin_bit_cast(v4f, a), y = __builtin_bit_cast(v4f, b);
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[j], y[j], c, 0, 0, 0);
  }
}
// row of value i of a lane's 16 (its column is the lane modulo 32)
DEV int row_of_acc(int i, int lane) { return 8 * (i / 4) + 4 * (lane / 32) + i % 4; }

// What a wave does with 32 by 32 of results of the lanes' rows and columns.  GATED: of the gate's and of the other product's at once.
template <typename T, int ACT> DEV void put_gated(const GemmArgs& p, int64_t m, int64_t n, float g, float u) {
  if (m >= p.M || n >= p.N) return;
  static_cast<T*>(p.c0)[m * p.sc0 + n] = from_f32<T>(act<ACT>(g) * u);
  if (p.pre) {
    p.pre[m * 2 * p.N + n] = g;
    p.pre[m * 2 * p.N + p.N + n] = u;
  }
}
template <typename T> DEV void put_plain(const GemmArgs& p, int64_t m, int64_t n, float v) {
  if (m >= p.M || n >= p.N) return;
  T* c = m < p.split ? static_cast<T*>(p.c0) + m * p.sc0 : static_cast<T*>(p.c1) + (m - p.split) * p.sc1;
  c[n] = from_f32<T>(v);
}

// ---- any alignment and size ----
// A workgroup of four waves forms 128 by BN of C (forward: 128 by BN / 2 of both products), each wave 64 by BN / 2.  The next tile's
// rows are in registers while this one is multiplied from shared memory; its 16-byte pieces are exchanged within a row by
// half of the row's number, so that no two of the sixteen lanes that read together meet in a bank.  Rows past the end are read as the last.  With
// p.parts > 1 the workgroups split k, and each writes float32 sums of its own to p.sums, [parts][M][N].
//
// Float32.  The matrix units multiply bfloat16 16 times as fast as float32.  A float32 is the exact sum of three bfloat16, each
// the nearest to what those before it leave: the second is at most 2^-8 of the value and the third 2^-16, of either sign.  Of the nine
// products of two such numbers six are formed, exactly, and summed in float32 like any product's terms; the three left out
// are 2^-24 of a term each at most, 2^-24 together in what was measured, and without a bias.  (Cut off and not rounded the parts have the
// value's sign and twice the size: what was left out reached 2^-21 and shrank every term, by 0.7 2^-24 on average.)  That is float32's
// accuracy at 2.7 times its rate: 6 instructions of 32 cycles in place of 8 of 64.  (An infinity less itself is a NaN: a
// float32 infinity makes its row's or column's results NaN here, infinite where few rows are multiplied in float32.)
template <typename T> struct Parts {
  static constexpr int PL = sizeof(T) == 4 ? 3 : 1;             // numbers that make one
  static constexpr int CPR = sizeof(T) == 4 ? 4 : 8;            // 16-byte pieces of a row in shared memory
  static DEV int swap(int r, int c) { return CPR == 8 ? c ^ (r >> 1 & 7) : c ^ (r >> 2 & 3); }
};
// two values as bfloat16, each to the nearest, in one instruction
DEV uint32_t pair_bf16(float a, float b) {
  using v2f = float __attribute__((ext_vector_type(2)));
  using v2b = __bf16 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v2f{a, b}, v2b));
}
DEV void split3(const v4u& x, uint32_t (&hi)[2], uint32_t (&mid)[2], uint32_t (&lo)[2]) {
  constexpr float most = 3.3895313892515355e38f;                // bfloat16's largest value: no finite value becomes an infinity
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float v[2], r[2], q[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) v[k] = __uint_as_float(x[2 * i + k]);
    hi[i] = pair_bf16(__builtin_amdgcn_fmed3f(v[0], -most, most), __builtin_amdgcn_fmed3f(v[1], -most, most));
    r[0] = v[0] - __uint_as_float(hi[i] << 16), r[1] = v[1] - __uint_as_float(hi[i] & 0xffff0000u);
    mid[i] = pair_bf16(r[0], r[1]);
    q[0] = r[0] - __uint_as_float(mid[i] << 16), q[1] = r[1] - __uint_as_float(mid[i] & 0xffff0000u);
    lo[i] = pair_bf16(q[0], q[1]);
  }
}
// 16 bytes that a thread has loaded (piece c of the 8 of row r) to shared memory of ROWS rows
template <typename T, int ROWS> DEV void put16(v4u (*to)[ROWS][Parts<T>::CPR], int r, int c, const v4u& v) {
  if constexpr (sizeof(T) == 2) {
    to[0][r][Parts<T>::swap(r, c)] = v;
  } else {
    uint32_t part[3][2];
    split3(v, part[0], part[1], part[2]);
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      using v2u = uint32_t __attribute__((ext_vector_type(2)));
      reinterpret_cast<v2u*>(&to[k][r][Parts<T>::swap(r, c / 2)])[c & 1] = v2u{part[k][0], part[k][1]};
    }
  }
}
template <typename T, int BN, bool GATED, int ACT>
__global__ __launch_bounds__(256) void k_gemm(const GemmArgs p, uint32_t mtiles, uint32_t tiles) {
  constexpr int V = 16 / sizeof(T), BK = kKBytes / sizeof(T), NF = BN / 64;   // NF: 32-column pieces of a wave
  constexpr int PL = Parts<T>::PL, CPR = Parts<T>::CPR;
  static_assert(BN == 64 || BN == 128, "pieces of 32 columns for two waves");
  __shared__ v4u sa[PL][128][CPR], sb[PL][BN][CPR];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave & 1, wn = wave >> 1;
  const uint32_t part = blockIdx.x / tiles, tile = blockIdx.x - part * tiles;
  const int64_t mt = tile % mtiles, nt = tile / mtiles;
  const int64_t m0 = mt * 128, n0 = nt * (GATED ? BN / 2 : BN);
  const int64_t k_begin = part * p.per_part, k_end = k_begin + p.per_part < p.K ? k_begin + p.per_part : p.K;
  const T* a = static_cast<const T*>(p.a);
  v4u ra[4], rb[BN / 32];
  const auto load = [&](int64_t k0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int id = threadIdx.x + i * 256, r = id / 8, c = id % 8;
      ra[i] = load16<T>(a + at_most(m0 + r, p.M - 1) * p.sa, k0 + c * V, k_end);
    }
    const int64_t past = !GATED && PL == 1 && k0 >= p.Kb ? p.Kb : 0;      // Kb is a multiple of BK then
#pragma unroll
    for (int i = 0; i < BN / 32; ++i) {
      const int id = threadIdx.x + i * 256, r = id / 8, c = id % 8;
      const bool second = GATED && r >= BN / 2;
      const int64_t n = at_most(n0 + (second ? r - BN / 2 : r), p.N - 1);
      const T* b = static_cast<const T*>(second ? p.b1 : p.b0);
      rb[i] = load16<T>(b + n * (second ? p.sb1 : p.sb0), k0 - past + c * V, k_end - past);
    }
  };
  v16f acc[2][NF] = {};
  load(k_begin);
  for (int64_t k0 = k_begin; k0 < k_end; k0 += BK) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int id = threadIdx.x + i * 256, r = id / 8, c = id % 8;
      put16<T, 128>(sa, r, c, ra[i]);
      if (i < BN / 32) put16<T, BN>(sb, r, c, rb[i < BN / 32 ? i : 0]);
    }
    __syncthreads();
    if (k0 + BK < k_end) load(k0 + BK);
#pragma unroll
    for (int kk = 0; kk < CPR / 2; ++kk) {
      v4u fa[2][PL], fb[NF][PL];
      const int c = kk * 2 + lane / 32;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = wm * 64 + i * 32 + (lane & 31);
#pragma unroll
        for (int q = 0; q < PL; ++q) fa[i][q] = sa[q][r][Parts<T>::swap(r, c)];
      }
#pragma unroll
      for (int j = 0; j < NF; ++j) {
        // gated, two pieces: 32 columns of the gate, then the same of the other product; one piece: 16 of each
        const int n = GATED ? (NF == 2 ? j * 64 + wn * 32 + (lane & 31) : (lane >> 4 & 1) * 32 + wn * 16 + (lane & 15))
                            : wn * (BN / 2) + j * 32 + (lane & 31);
#pragma unroll
        for (int q = 0; q < PL; ++q) fb[j][q] = sb[q][n][Parts<T>::swap(n, c)];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          // the small products first
          if constexpr (PL == 3) {
            mma<bf16>(fa[i][2], fb[j][0], acc[i][j]);
            mma<bf16>(fa[i][0], fb[j][2], acc[i][j]);
            mma<bf16>(fa[i][1], fb[j][1], acc[i][j]);
            mma<bf16>(fa[i][1], fb[j][0], acc[i][j]);
            mma<bf16>(fa[i][0], fb[j][1], acc[i][j]);
          }
          mma<bf16>(fa[i][0], fb[j][0], acc[i][j]);
        }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int64_t m = m0 + wm * 64 + i * 32 + row_of_acc(e, lane);
      if constexpr (GATED && NF == 2) {
        put_gated<T, ACT>(p, m, n0 + wn * 32 + (lane & 31), acc[i][0][e], acc[i][1][e]);
      } else if constexpr (GATED) {
        const float u = __shfl_xor(acc[i][0][e], 16);      // of the lane with the same column of the other product
        if (!(lane & 16)) put_gated<T, ACT>(p, m, n0 + wn * 16 + (lane & 15), acc[i][0][e], u);
      } else {
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          const int64_t n = n0 + wn * (BN / 2) + j * 32 + (lane & 31);
          if (p.parts > 1) {
            if (m < p.M && n < p.N) p.sums[(part * p.M + m) * p.N + n] = acc[i][j][e];
          } else {
            put_plain<T>(p, m, n, acc[i][j][e]);
          }
        }
      }
    }
}
// C from the parts' sums, added in order
template <typename T> __global__ __launch_bounds__(256) void k_join(const GemmArgs p) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, size = p.M * p.N;
  if (i >= size) return;
  float s = p.sums[i];
  for (int32_t k = 1; k < p.parts; ++k) s += p.sums[k * size + i];
  const int64_t m = i / p.N;
  put_plain<T>(p, m, i - m * p.N, s);
}

// ---- large, aligned, bfloat16 ----
// 256 by 256 of C (forward: 256 by 128 of both products) a workgroup of eight waves, two by four, each 128 by 64 with its sums in 128
// registers, two waves a SIMD.  Two stages of 128 bytes of k lie in shared memory: the loads go there past the registers, those of one
// stage while the other is multiplied.  (Four stages of 64 bytes ask for every cache line twice, and the cache between has forgotten
// it by then.)  A load puts down its lanes' 16 bytes in a row, so the exchange that keeps reads off each other's banks (the pieces of
// sixteen rows fill 256 bytes twice over where they are exchanged by a row's number, once by half of it) is made by which piece each
// lane asks for.  Reads and loads are issued between the products, each of which keeps the matrix unit busy for eight instructions'
// time.  Eight waves against four of 128 by 128 (one a SIMD, so that a wait is a stall), forward with pre: R = D = F = 2048 54 and 61 us,
// R = 4096, D = 1024, F = 4096 80 and 90, R = 8192, D = 4096, F = 8192 (1.1 TFLOP) 1018 and 1007, gradient 2126 and 2186 (with
// one bfloat16 for each of dg and du; with two it is 3820: 1675 us for each of its products, 1.31 PFLOP/s, 77% of the matrix units' time).
// Rows past the end are read as the last and left out of the result.  k is a multiple of the stage, everything 16-byte
// aligned.  Neighbouring tiles share rows and columns: each of the eight L2 caches gets a run of tiles of its own, in bands of
// eight rows of tiles.
constexpr int kStages = 2, kStageBytes = 512 * 128, kLoads = 8;   // loads of a thread for a stage
DEV void load_to_lds(const void* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from) : "memory", "m0");
}
// all loads have landed, all reads of the past stage are done, in every wave
DEV void stage_ready() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
template <int FROM, int TO, typename F> DEV void unrolled(F&& f) {
  if constexpr (FROM < TO) {
    f(std::integral_constant<int, FROM>{});
    unrolled<FROM + 1, TO>(f);
  }
}
template <bool GATED, int ACT>
__global__ __launch_bounds__(512, 2) void k_gemm_large(const GemmArgs p, uint32_t mtiles, uint32_t ntiles) {
  using T = bf16;
  constexpr int BK = 128 / sizeof(T);
  __shared__ __attribute__((aligned(128))) char smem[kStages * kStageBytes];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave & 1, wn = wave >> 1;
  // the tile: a run of tiles for each XCD (the block number modulo 8), in bands
  const uint32_t tiles = mtiles * ntiles, xcd = blockIdx.x & 7, q = tiles >> 3, r8 = tiles & 7;
  const uint32_t id = xcd * q + (xcd < r8 ? xcd : r8) + (blockIdx.x >> 3);
  const uint32_t band = id / (8 * ntiles), in = id - band * (8 * ntiles), rows = mtiles - band * 8 < 8 ? mtiles - band * 8 : 8;
  const int64_t m0 = static_cast<int64_t>(band * 8 + in % rows) * 256, n0 = static_cast<int64_t>(in / rows) * (GATED ? 128 : 256);

  // wave w loads the rows w 32 .. w 32 + 31 of A and of B, 8 a load: lane l puts down piece l % 8 of row l / 8
  const T* from[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = wave * 32 + (i & 3) * 8 + lane / 8, c = (lane & 7) ^ (r >> 1 & 7);
    if (i < 4) {
      from[i] = static_cast<const T*>(p.a) + at_most(m0 + r, p.M - 1) * p.sa + c * (16 / sizeof(T));
    } else {
      const bool second = GATED && r >= 128;
      const int64_t n = at_most(n0 + (second ? r - 128 : r), p.N - 1);
      from[i] = static_cast<const T*>(second ? p.b1 : p.b0) + n * (second ? p.sb1 : p.sb0) + c * (16 / sizeof(T));
    }
  }
  const uint32_t base = static_cast<uint32_t>((uintptr_t)(__attribute__((address_space(3))) char*)smem) + wave * 4096;   // in the LDS
  const int count = static_cast<int>(p.K / BK), half = lane / 32, l32 = lane & 31;
  // stage n's way to the next one: nowhere behind the last, which is loaded again, so that nothing branches; B's may begin anew
  const int again = GATED ? 0 : static_cast<int>(p.Kb / BK);
  const auto step_a = [&](int n) -> int64_t { return n + 1 < count ? BK : 0; };
  const auto step_b = [&](int n) -> int64_t { return n + 1 >= count ? 0 : !GATED && n + 1 == again ? BK - p.Kb : BK; };
  // stage n, which is next, to its place
  const auto load = [&](int stage, int n, auto which) {
    constexpr int i = which;
    load_to_lds(from[i], base + stage * kStageBytes + (i >> 2) * 32768 + (i & 3) * 1024);
    from[i] += i < 4 ? step_a(n) : step_b(n);
  };
  v16f acc[4][2] = {};
  struct Pieces { v4u a[4], b[2]; };
  const auto read = [&](int stage, int kk, Pieces& f, auto which) {
    constexpr int i = which;
    const v4u* at = reinterpret_cast<const v4u*>(smem + stage * kStageBytes);
    const int c = kk * 2 + half;
    if constexpr (i < 4) {
      const int r = wm * 128 + i * 32 + l32;
      f.a[i] = at[r * 8 + (c ^ (r >> 1 & 7))];
    } else {
      // gated: 32 columns of the gate, then the same of the other product
      constexpr int j = i - 4;
      const int n = GATED ? j * 128 + wn * 32 + l32 : wn * 64 + j * 32 + l32;
      f.b[j] = at[256 * 8 + n * 8 + (c ^ (n >> 1 & 7))];
    }
  };
  // the products of f, `beside(k)` after the k-th of the sixteen
  const auto multiply = [&](const Pieces& f, auto&& beside) {
    unrolled<0, 8>([&](auto which) {
      constexpr int k = which;
      mma<T>(f.a[k >> 1], f.b[k & 1], acc[k >> 1][k & 1]);
      beside(which);
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  // quarter kk of a stage, with the reads of the next one beside it
  const auto quarter = [&](int stage, int kk, const Pieces& f, Pieces& next) {
    multiply(f, [&](auto which) {
      constexpr int k = which;
      if constexpr (k < 6) read(stage, kk + 1, next, which);
    });
  };
  Pieces even, odd;
  unrolled<0, kLoads>([&](auto i) { load(0, 0, i); });
  stage_ready();
  unrolled<0, kLoads>([&](auto i) { load(1, 1, i); });
  unrolled<0, 6>([&](auto i) { read(0, 0, even, i); });
#pragma unroll 1
  for (int k = 0; k < count; ++k) {
    const int stage = k & 1;
    quarter(stage, 0, even, odd);
    quarter(stage, 1, odd, even);
    quarter(stage, 2, even, odd);
    // the last quarter's operands are in registers: when every wave is here, this stage's place is free, and the next one is there
    stage_ready();
    multiply(odd, [&](auto which) {
      constexpr int i = which;
      load(stage, k + 2, which);
      if constexpr (i < 6) read(stage ^ 1, 0, even, which);
    });
  }
  stage_ready();                // nothing is on its way to shared memory when the workgroup ends
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int64_t m = m0 + wm * 128 + i * 32 + row_of_acc(e, lane);
#pragma unroll
      for (int j = 0; j < (GATED ? 1 : 2); ++j) {
        if constexpr (GATED) put_gated<T, ACT>(p, m, n0 + wn * 32 + l32, acc[i][0][e], acc[i][1][e]);
        else put_plain<T>(p, m, n0 + wn * 64 + j * 32 + l32, acc[i][j][e]);
      }
    }
}

// ---- few rows ----
// The weights are read once: a workgroup has 16 columns of the gate and the same 16 of the other product side by side, and its eight
// waves take every eighth 128 bytes of k, each by itself; their sums meet in shared memory.  MT: 32-row pieces of x.  Rows
// beyond MT 32 are for other workgroups, eight blocks on (the same XCD), which read the weights again.
constexpr int kFewWaves = 8;
struct FewPlace {
  int64_t f0, m0;
};
DEV FewPlace few_place(uint32_t groups, int rows) {
  const uint32_t turn = blockIdx.x >> 3;
  return {(static_cast<int64_t>(turn / groups) * 8 + (blockIdx.x & 7)) * 16, static_cast<int64_t>(turn % groups) * rows};
}
// row r of the 32 of both weights
template <typename T> DEV const T* few_weight(const GemmArgs& p, int64_t f0, int r) {
  const int64_t f = at_most(f0 + (r & 15), p.N - 1);
  return r < 16 ? static_cast<const T*>(p.b0) + f * p.sb0 : static_cast<const T*>(p.b1) + f * p.sb1;
}
// part: [waves][MT 32][33] floats; 33: rows of 32 begin in banks of their own
template <typename T, int MT, int ACT> DEV void few_join(const GemmArgs& p, float* part, const v16f (&acc)[MT], const FewPlace& at) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) part[((wave * MT + i) * 32 + row_of_acc(e, lane)) * 33 + (lane & 31)] = acc[i][e];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = i * 32 + (threadIdx.x >> 4), c = threadIdx.x & 15;
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int k = 0; k < kFewWaves; ++k) {
      g += part[(k * MT * 32 + m) * 33 + c];
      u += part[(k * MT * 32 + m) * 33 + c + 16];
    }
    put_gated<T, ACT>(p, at.m0 + m, at.f0 + c, g, u);
  }
}

// Any alignment: from global memory straight into the matrix operands.  A lane reads 64 bytes of its row's 128, four pieces that are
// four steps of k, x's rows alike; so a load asks for 64 cache lines, and these bound it.
template <typename T, int MT, int ACT>
__global__ __launch_bounds__(512) void k_few_rows(const GemmArgs p, uint32_t groups) {
  constexpr int V = 16 / sizeof(T), BK = kKBytes / sizeof(T);
  __shared__ float part[kFewWaves * MT * 32 * 33];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l32 = lane & 31, half = lane / 32;
  const FewPlace at = few_place(groups, MT * 32);
  if (at.f0 >= p.N) return;
  const T* w = few_weight<T>(p, at.f0, l32);
  const T* x[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) x[i] = static_cast<const T*>(p.a) + at_most(at.m0 + i * 32 + l32, p.M - 1) * p.sa;
  v4u rw[2][4], rx[2][MT][4];
  const auto load = [&](int64_t k0, v4u (&bw)[4], v4u (&bx)[MT][4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t k = k0 + (half * 4 + j) * V;
      bw[j] = load16<T>(w, k, p.K);
#pragma unroll
      for (int i = 0; i < MT; ++i) bx[i][j] = load16<T>(x[i], k, p.K);
    }
  };
  v16f acc[MT] = {};
  const auto multiply = [&](const v4u (&bw)[4], const v4u (&bx)[MT][4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < MT; ++i) mma<T>(bx[i][j], bw[j], acc[i]);
  };
  int64_t k = static_cast<int64_t>(wave) * BK;
  constexpr int64_t STEP = kFewWaves * BK;
  if (k < p.K) load(k, rw[0], rx[0]);
  for (; k < p.K; k += 2 * STEP) {
    if (k + STEP < p.K) load(k + STEP, rw[1], rx[1]);
    multiply(rw[0], rx[0]);
    if (k + STEP >= p.K) break;
    if (k + 2 * STEP < p.K) load(k + 2 * STEP, rw[0], rx[0]);
    multiply(rw[1], rx[1]);
  }
  few_join<T, MT, ACT>(p, part, acc, at);
}

// k in whole 128 bytes, everything 16-byte aligned: each wave's weights and rows of x go to two places of its own in shared memory,
// past the registers, eight whole cache lines a load; no wave waits for another.  32 rows, bf16, D = 4096, F = 8192: 29 us, 4.6 TB/s
// of weights (a copy runs at 5.06), against 52 straight into the operands.
template <typename T, int ACT>
__global__ __launch_bounds__(512) void k_few_rows_aligned(const GemmArgs p, uint32_t groups) {
  constexpr int MT = 1, BK = kKBytes / sizeof(T), ROWS = 32 * (1 + MT), LOADS = ROWS / 8, PLACE = ROWS * 128;
  __shared__ __attribute__((aligned(128))) char smem[kFewWaves * 2 * PLACE];
  static_assert(sizeof(smem) >= kFewWaves * MT * 32 * 33 * sizeof(float), "the sums meet in the same place");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l32 = lane & 31, half = lane / 32;
  const FewPlace at = few_place(groups, MT * 32);
  if (at.f0 >= p.N) return;
  // load i: rows 8 i .. 8 i + 7 of the weights' 32, then of x's; lane l puts down piece l % 8 of row l / 8, exchanged as above
  const T* from[LOADS];
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const int r = i * 8 + lane / 8;
    const T* row = i < 4 ? few_weight<T>(p, at.f0, r) : static_cast<const T*>(p.a) + at_most(at.m0 + r - 32, p.M - 1) * p.sa;
    from[i] = row + static_cast<int64_t>(wave) * BK + ((lane & 7) ^ (r >> 1 & 7)) * (16 / sizeof(T));
  }
  char* own = smem + wave * 2 * PLACE;
  const uint32_t base = static_cast<uint32_t>((uintptr_t)(__attribute__((address_space(3))) char*)own);
  const auto load = [&](int place) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      load_to_lds(from[i], base + place * PLACE + i * 1024);
      from[i] += kFewWaves * BK;
    }
  };
  const int blocks = static_cast<int>(p.K / BK), count = wave < blocks ? (blocks - wave + kFewWaves - 1) / kFewWaves : 0;
  v16f acc[MT] = {};
  if (count > 0) load(0);
  if (count > 1) load(1);
  for (int k = 0; k < count; ++k) {
    // this place's loads have landed; those of the other one, if any, are behind them
    if (k + 1 < count) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LOADS) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const v4u* rows = reinterpret_cast<const v4u*>(own + (k & 1) * PLACE);
    v4u fw[4], fx[MT][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = (j * 2 + half) ^ (l32 >> 1 & 7);
      fw[j] = rows[l32 * 8 + c];
#pragma unroll
      for (int i = 0; i < MT; ++i) fx[i][j] = rows[((1 + i) * 32 + l32) * 8 + c];
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");          // what was read here may be written over
    if (k + 2 < count) load(k & 1);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < MT; ++i) mma<T>(fx[i][j], fw[j], acc[i]);
  }
  __syncthreads();
  few_join<T, MT, ACT>(p, reinterpret_cast<float*>(smem), acc, at);
}

// ---------------- what the gradients' products are made of ----------------
// 64 by 64 values that go through shared memory to be written along their other dimension, 16 bytes a lane both ways.  Rows of an
// odd number of words: the eight lanes that gather eight rows each, and the words of their columns, fall into banks of their own.
template <typename T> struct Turn {
  static constexpr int V = 16 / sizeof(T), PER = 64 / V, N = 64 * PER / 256;   // pieces of a row; pieces of a thread
  static constexpr int ROW = 64 * sizeof(T) / 4 + 1;
  uint32_t w[64 * ROW];
  DEV void put(int r, int c, const v4u& v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[r * ROW + c * 4 + i] = v[i];
  }
  // column c, rows V k .. V k + V - 1
  DEV v4u get(int c, int k) const {
    v4u v;
    if constexpr (sizeof(T) == 2) {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(w);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = h[(k * 8 + 2 * i) * ROW * 2 + c] | static_cast<uint32_t>(h[(k * 8 + 2 * i + 1) * ROW * 2 + c]) << 16;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = w[(k * 4 + i) * ROW + c];
    }
    return v;
  }
};
// the first n elements of 16 bytes
template <typename T> DEV void store16(T* p, int64_t n, const v4u& v) {
  constexpr int V = 16 / sizeof(T);
  if (n >= V) {
    LooseWords<T, V> q;
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = v[i];
    *reinterpret_cast<LooseWords<T, V>*>(p) = q;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) {
        if constexpr (sizeof(T) == 2) p[i].u = static_cast<uint16_t>(v[i / 2] >> (i % 2 * 16));
        else p[i] = __uint_as_float(v[i]);
      }
  }
}

// A float32 as the sum of two bfloat16, off by 2^-16 of it at most: dg and du, which the matrix units multiply in bfloat16.  (One
// bfloat16 would put d_x and d_w off by 2.3e-3 where their own rounding is 1.7e-3.)  Finite values stay finite, infinities are the first's.
template <int V> DEV void two_bf16(float (&x)[V], Vec<bf16, V>& first, Vec<bf16, V>& rest) {
  constexpr float most = 3.3895313892515355e38f;                // bfloat16's largest value
  float r[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float a = fabsf(x[i]);
    r[i] = x[i];
    if (a > most && a < __builtin_huge_valf()) x[i] = copysignf(most, x[i]);
  }
  first = pack_vec<bf16, V>(x);
#pragma unroll
  for (int i = 0; i < V; ++i) r[i] = fabsf(r[i]) < __builtin_huge_valf() ? r[i] - first.get(i) : 0.0f;
  rest = pack_vec<bf16, V>(r);
}

// dg and du of R rows as [R][F2] and as [2 F][Rp], zeros from 2 F to F2 and from R to Rp; 64 by 64 of each a workgroup.  In bfloat16
// two planes of each, side by side in a row: [R][2][F2] and [2 F][2][Rp].
struct SplitArgs {
  const float* pre;
  const void* dh;
  int64_t sdh, R, F;
  int64_t Rp, Rs, F2, Fs;       // lengths of a plane's row of `cols` and of `rows` with their zeros, and row strides
  void *rows, *cols;
};
template <typename T, int ACT> __global__ __launch_bounds__(256) void k_ffn_split(const SplitArgs p, uint32_t ftiles) {
  using L = Turn<T>;
  constexpr int PL = planes_of(sizeof(T));
  __shared__ L tg[PL], tu[PL];
  // neighbouring workgroups take neighbouring columns: rows may lie a large power of two apart, in few of the memory's channels
  const int64_t r0 = static_cast<int64_t>(blockIdx.x / ftiles) * 64, f0 = static_cast<int64_t>(blockIdx.x % ftiles) * 64;
#pragma unroll
  for (int k = 0; k < L::N; ++k) {
    const int id = threadIdx.x + k * 256, i = id / L::PER, c = id % L::PER;
    const int64_t r = r0 + i, f = f0 + c * L::V, n = r < p.R ? p.F - f : 0;
    const float* pre = p.pre + r * 2 * p.F + f;
    const Vec<T, L::V> vh = load_row<T, L::V, true>(static_cast<const T*>(p.dh) + r * p.sdh + f, n, T{});
    float dg[L::V], du[L::V];
#pragma unroll
    for (int h = 0; h < L::V; h += 4) {
      const Vec<float, 4> vg = load_row<float, 4, true>(pre + h, n - h, 0.0f), vu = load_row<float, 4, true>(pre + p.F + h, n - h, 0.0f);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float g = vg.get(e), dh = vh.get(h + e);
        dg[h + e] = dh * vu.get(e) * slope<ACT>(g);
        du[h + e] = dh * act<ACT>(g);
      }
    }
    Vec<T, L::V> og[PL], ou[PL];
    if constexpr (PL == 2) {
      two_bf16<L::V>(dg, og[0], og[1]);
      two_bf16<L::V>(du, ou[0], ou[1]);
    } else {
      og[0] = pack_vec<T, L::V>(dg);
      ou[0] = pack_vec<T, L::V>(du);
    }
#pragma unroll
    for (int q = 0; q < PL; ++q) {
      const v4u bg{og[q].w[0], og[q].w[1], og[q].w[2], og[q].w[3]}, bu{ou[q].w[0], ou[q].w[1], ou[q].w[2], ou[q].w[3]};
      if (p.rows && n > 0) {
        T* to = static_cast<T*>(p.rows) + r * p.Fs + q * p.F2 + f;
        store16<T>(to, n, bg);
        store16<T>(to + p.F, n, bu);
      }
      if (p.cols) {
        tg[q].put(i, c, bg);
        tu[q].put(i, c, bu);
      }
    }
  }
  if (p.rows && f0 == 0) {                                      // k's padding
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = 0; i < 16 && r0 + wave * 16 + i < p.R; ++i)
      if (2 * p.F + lane < p.F2)
#pragma unroll
        for (int q = 0; q < PL; ++q) static_cast<T*>(p.rows)[(r0 + wave * 16 + i) * p.Fs + q * p.F2 + 2 * p.F + lane] = T{};
  }
  if (!p.cols) return;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < L::N; ++k) {
    const int id = threadIdx.x + k * 256, c = id / L::PER, v = id % L::PER;
    const int64_t f = f0 + c, r = r0 + v * L::V;
    if (f < p.F) {
#pragma unroll
      for (int q = 0; q < PL; ++q) {
        T* to = static_cast<T*>(p.cols) + f * p.Rs + q * p.Rp + r;
        store16<T>(to, p.Rp - r, tg[q].get(c, v));
        store16<T>(to + p.F * p.Rs, p.Rp - r, tu[q].get(c, v));
      }
    }
  }
}

// to[c][r] = from[r][c] for R rows of C, zeros for r from R to Rp; `to` has row stride st
template <typename T>
__global__ __launch_bounds__(256) void k_transpose(const T* from, int64_t sf, int64_t R, int64_t C, T* to, int64_t st, int64_t Rp,
                                                   uint32_t ctiles) {
  using L = Turn<T>;
  __shared__ L tile;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x / ctiles) * 64, c0 = static_cast<int64_t>(blockIdx.x % ctiles) * 64;
#pragma unroll
  for (int k = 0; k < L::N; ++k) {
    const int id = threadIdx.x + k * 256, i = id / L::PER, c = id % L::PER;
    const int64_t r = r0 + i;
    tile.put(i, c, load16<T>(from + r * sf, c0 + c * L::V, r < R ? C : 0));
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < L::N; ++k) {
    const int id = threadIdx.x + k * 256, c = id / L::PER, q = id % L::PER;
    const int64_t r = r0 + q * L::V;
    if (c0 + c < C) store16<T>(to + (c0 + c) * st + r, Rp - r, tile.get(c, q));
  }
}

// ---------------- host ----------------
inline int64_t padded(int64_t n) { return ceil_div(n, kPad) * kPad; }
constexpr int64_t kCus = 256, kMostParts = 8;
// Whether the large tiles are for C of M by N (forward: by 2 N): they have to fill half of the chip.  Forward, D = 1024, bf16: 64 of them
// (R = 1024, F = 2048) 27 us and 20 in k_gemm's, 128 (F = 4096) 30 and 34, 256 (R = 2048) 37 and 54.
static bool large(int64_t M, int64_t N, bool gated) { return ceil_div(M, 256) * ceil_div(N, gated ? 128 : 256) >= kCus / 2; }
static bool aligned16(const void* p, int64_t stride, size_t e) { return aligned(p, 16) && stride * static_cast<int64_t>(e) % 16 == 0; }
// Columns of a workgroup of k_gemm: 128 where those workgroups are twice the chip's units, or once for two products in bfloat16.
// Whole calls with 128 and 64, float32: gradient of 387 (R = 1001, D = 1025, F = 2731) 235 and 216 us, 512 (R = 700, D = 1024, F = 4096)
// 196 and 208; forward with pre 344 (the first) 85 and 89, 512 (R = 1024) 103 and 116; bfloat16 344 (the first) 32 and 37, 384 27 and 30.
// (bfloat16 gradients of so many are in the large tiles: 256, R = 1500, D = 1000, F = 2000, took 138 us with 128 columns, 125 with 64.)
static int columns_of(size_t e, int64_t M, int64_t N, bool gated) {
  if (e == 2 && !gated) return 64;
  return ceil_div(M, 128) * ceil_div(N, gated ? 64 : 128) >= (e == 2 ? kCus : 2 * kCus) ? 128 : 64;
}
// parts of k: they fill the chip three times (twice, four and six times make no difference)
static int64_t parts_of(size_t e, int64_t M, int64_t N, int64_t K) {
  const int64_t tiles = ceil_div(M, 128) * ceil_div(N, columns_of(e, M, N, false)), most = K * static_cast<int64_t>(e) / (8 * kKBytes);
  if (tiles == 0) return 1;
  return std::max<int64_t>(1, std::min({3 * kCus / tiles, most, kMostParts}));
}

template <typename T, int BN, bool GATED, int ACT> static bool gemm_of(const GemmArgs& p, hipStream_t st) {
  const int64_t mt = ceil_div(p.M, 128), nt = ceil_div(p.N, GATED ? BN / 2 : BN);
  if (!grid_ok(mt * nt * p.parts, 256)) return false;
  k_gemm<T, BN, GATED, ACT><<<dim3(static_cast<uint32_t>(mt * nt * p.parts)), dim3(256), 0, st>>>(
      p, static_cast<uint32_t>(mt), static_cast<uint32_t>(mt * nt));
  return true;
}
// `sums`: room for parts_of() M N floats, or null for one part
template <typename T, bool GATED, int ACT> static bool gemm(GemmArgs p, float* sums, hipStream_t st) {
  if (p.M == 0 || p.N == 0) return true;
  const size_t e = sizeof(T);
  p.parts = 1;
  p.per_part = p.K;
  if constexpr (sizeof(T) == 2) if (large(p.M, p.N, GATED) && p.K > 0 && p.K * static_cast<int64_t>(e) % kKBytes == 0 &&
      aligned16(p.a, p.sa, e) && aligned16(p.b0, p.sb0, e) && (!GATED || aligned16(p.b1, p.sb1, e))) {
    const int64_t mt = ceil_div(p.M, 256), nt = ceil_div(p.N, GATED ? 128 : 256);
    if (!grid_ok(mt * nt, 512)) return false;
    k_gemm_large<GATED, ACT><<<dim3(static_cast<uint32_t>(mt * nt)), dim3(512), 0, st>>>(
        p, static_cast<uint32_t>(mt), static_cast<uint32_t>(nt));
    return true;
  }
  if (sums) {
    const int64_t parts = parts_of(e, p.M, p.N, p.K), bk = kKBytes / e;
    p.sums = sums;
    p.per_part = ceil_div(ceil_div(p.K, parts), bk) * bk;
    p.parts = p.K ? static_cast<int32_t>(ceil_div(p.K, p.per_part)) : 1;
  }
  bool wide = false, ok = true;
  if constexpr (GATED || sizeof(T) == 4) {
    wide = columns_of(e, p.M, p.N, GATED) == 128;
    if (wide) ok = gemm_of<T, 128, GATED, ACT>(p, st);
  }
  if (!wide) ok = gemm_of<T, 64, GATED, ACT>(p, st);
  if (!ok) return false;
  if (p.parts > 1) {
    const int64_t blocks = ceil_div(p.M * p.N, 256);
    if (!grid_ok(blocks, 256)) return false;
    k_join<T><<<dim3(static_cast<uint32_t>(blocks)), dim3(256), 0, st>>>(p);
  }
  return true;
}
// k in whole 128 bytes and everything 16-byte aligned
template <typename T> static bool whole(const GemmArgs& p) {
  return p.K > 0 && p.K * static_cast<int64_t>(sizeof(T)) % kKBytes == 0 && aligned16(p.a, p.sa, sizeof(T)) &&
         aligned16(p.b0, p.sb0, sizeof(T)) && aligned16(p.b1, p.sb1, sizeof(T));
}
template <typename T, int MT, int ACT> static bool few_rows(const GemmArgs& p, hipStream_t st) {
  const bool w = whole<T>(p);
  const int64_t groups = ceil_div(p.M, w ? 32 : MT * 32), blocks = ceil_div(ceil_div(p.N, 16), 8) * 8 * groups;
  if (!grid_ok(blocks, 512)) return false;
  const dim3 grid(static_cast<uint32_t>(blocks));
  if (w) k_few_rows_aligned<T, ACT><<<grid, dim3(512), 0, st>>>(p, static_cast<uint32_t>(groups));
  else k_few_rows<T, MT, ACT><<<grid, dim3(512), 0, st>>>(p, static_cast<uint32_t>(groups));
  return true;
}
// Up to which row count the weights are streamed past few rows.  bf16, D = 4096, F = 8192: 64, 96, 128 rows 44, 63, 80 us, 129 in tiles
// 75; D = 1024, F = 4096: 128 rows 13.6 us, 129 in tiles 18.0.  Float32, bound by its matrix instructions: 64 rows 115 us, 96
// in tiles 168.
template <typename T> static int64_t few_most(const GemmArgs& p) { return sizeof(T) == 2 && whole<T>(p) ? 128 : 64; }
template <typename T, int ACT> static bool forward(const GemmArgs& p, hipStream_t st) {
  if (p.M > few_most<T>(p)) return gemm<T, true, ACT>(p, nullptr, st);
  return p.M <= 32 ? few_rows<T, 1, ACT>(p, st) : few_rows<T, 2, ACT>(p, st);
}
template <typename T> static bool transpose(const void* from, int64_t sf, int64_t R, int64_t C, T* to, int64_t st, int64_t Rp,
                                            hipStream_t stream) {
  const int64_t rt = ceil_div(Rp, 64), ct = ceil_div(C, 64);
  if (rt == 0 || ct == 0) return true;
  if (!grid_ok(rt * ct, 256)) return false;
  k_transpose<T><<<dim3(static_cast<uint32_t>(rt * ct)), dim3(256), 0, stream>>>(static_cast<const T*>(from), sf, R, C, to, st, Rp,
                                                                                 static_cast<uint32_t>(ct));
  return true;
}

constexpr int64_t kMost = INT32_MAX - 512;
static bool sizes_ok(int64_t R, int64_t D, int64_t F) {
  return R >= 0 && D >= 0 && F >= 0 &&
         (R > kMost || D > kMost || F > kMost || (sizes_fit(R, D, 4) && sizes_fit(R, F, 4) && sizes_fit(F, D, 4)));
}
// Row stride of n elements in the workspace: not a large power of two, which would put the rows of a tile behind each other in few
// of the memory's channels (the two gradient products of R = 8192, D = 4096, F = 8192, with one bfloat16 for
// each of dg and du: 970 -> 882 us each).
static int64_t spread(int64_t n, size_t e) { return n * static_cast<int64_t>(e) % 4096 ? n : n + kPad; }
// elements of the gradient's workspace: d_pre [R][planes][F2], d_pre^T [2 F][planes][Rp], x^T [D][Rp], weights^T [D][F2], with row
// strides Fs, Rs, Xs and Ws, and float32 sums of parts of k
struct GradRoom {
  int64_t F2, Rp, Fs, Rs, Xs, Ws, rows, cols, xt, wt, sums;
  int64_t bytes(size_t e) const { return (rows + cols + xt + wt) * static_cast<int64_t>(e) + sums * 4; }
};
static GradRoom grad_room(size_t e, int64_t R, int64_t D, int64_t F) {
  GradRoom g;
  const int64_t n = planes_of(e);
  g.F2 = padded(2 * F), g.Rp = padded(R);
  const int64_t px = parts_of(e, R, D, n * g.F2), pw = parts_of(e, 2 * F, D, n * g.Rp);
  g.sums = std::max(px > 1 ? px * R * D : 0, pw > 1 ? pw * 2 * F * D : 0);
  g.Fs = spread(n * g.F2, e), g.Rs = spread(n * g.Rp, e), g.Xs = spread(g.Rp, e), g.Ws = spread(g.F2, e);
  g.rows = padded(R * g.Fs), g.cols = padded(2 * F * g.Rs), g.xt = padded(D * g.Xs), g.wt = padded(D * g.Ws);
  return g;
}

template <typename T, int ACT>
static pararnn_status backward(int64_t R, int64_t D, int64_t F, const void* x, int64_t sx, const void* wg, int64_t sg, const void* wu,
                               int64_t su, const float* pre, const void* dh, int64_t sdh, void* dx, int64_t sdx, void* dwg,
                               int64_t sdg, void* dwu, int64_t sdu, T* ws, hipStream_t st) {
  const GradRoom room = grad_room(sizeof(T), R, D, F);
  T *rows = ws, *cols = rows + room.rows, *xt = cols + room.cols, *wt = xt + room.xt;
  float* sums = reinterpret_cast<float*>(wt + room.wt);
  const int64_t rt = ceil_div(room.Rp, 64), ft = ceil_div(F, 64);
  if (!grid_ok(rt * ft, 256)) return PARARNN_ERR_UNSUPPORTED;
  bool ok = true;
  if (rt * ft) {
    const SplitArgs s{pre, dh, sdh, R, F, room.Rp, room.Rs, room.F2, room.Fs, dx ? rows : nullptr, dwg ? cols : nullptr};
    k_ffn_split<T, ACT><<<dim3(static_cast<uint32_t>(rt * ft)), dim3(256), 0, st>>>(s, static_cast<uint32_t>(ft));
  }
  if (dx && R && D) {
    ok = ok && transpose<T>(wg, sg, F, D, wt, room.Ws, F, st) && transpose<T>(wu, su, F, D, wt + F, room.Ws, room.F2 - F, st);
    const GemmArgs p{rows, wt, nullptr, room.Fs, room.Ws, 0, R, D, planes_of(sizeof(T)) * room.F2, room.F2, dx, nullptr, sdx, 0, R};
    ok = ok && gemm<T, false, 0>(p, room.sums ? sums : nullptr, st);
  }
  if (dwg && F && D) {
    ok = ok && transpose<T>(x, sx, R, D, xt, room.Xs, room.Rp, st);
    const GemmArgs p{cols, xt, nullptr, room.Rs, room.Xs, 0, 2 * F, D, planes_of(sizeof(T)) * room.Rp, room.Rp, dwg, dwu, sdg, sdu, F};
    ok = ok && gemm<T, false, 0>(p, room.sums ? sums : nullptr, st);
  }
  return ok ? launched() : PARARNN_ERR_UNSUPPORTED;
}

}  // namespace lm

using namespace lm;

extern "C" size_t pararnn_block_gated_linear_workspace_bytes(int dtype, int64_t R, int64_t D, int64_t F, int gradient) {
  if (!dtype_ok(dtype) || !sizes_ok(R, D, F) || R > kMost || D > kMost || F > kMost) return 0;
  return gradient ? static_cast<size_t>(grad_room(dtype_size(dtype), R, D, F).bytes(dtype_size(dtype))) : 0;
}

extern "C" pararnn_status pararnn_block_gated_linear(int dtype, int act, int64_t R, int64_t D, int64_t F, const void* x,
                                                     int64_t x_stride, const void* w_gate, int64_t gate_stride, const void* w_up,
                                                     int64_t up_stride, void* h, int64_t h_stride, float* pre, void* ws,
                                                     size_t ws_bytes, void* stream) {
  if (!dtype_ok(dtype) || (act != PARARNN_BLOCK_SILU && act != PARARNN_BLOCK_GELU) || !sizes_ok(R, D, F))
    return PARARNN_ERR_INVALID_ARG;
  const size_t e = dtype_size(dtype);
  if (!ptr_ok(x, e, R > 0 && D > 0) || !ptr_ok(w_gate, e, F > 0 && D > 0) || !ptr_ok(w_up, e, F > 0 && D > 0) ||
      !ptr_ok(h, e, R > 0 && F > 0) || !ptr_ok(pre, 4, false) || !plane_ok(R, x_stride) || !plane_ok(F, gate_stride) ||
      !plane_ok(F, up_stride) || !plane_ok(R, h_stride))
    return PARARNN_ERR_INVALID_ARG;
  if (R > kMost || D > kMost || F > kMost) return PARARNN_ERR_UNSUPPORTED;
  if (!ws_ok(ws, ws_bytes, pararnn_block_gated_linear_workspace_bytes(dtype, R, D, F, 0))) return PARARNN_ERR_WORKSPACE;
  if (R == 0 || F == 0) return PARARNN_OK;
  const GemmArgs p{x, w_gate, w_up, x_stride, gate_stride, up_stride, R, F, D, D, h, nullptr, h_stride, 0, R, pre, nullptr, D, 1};
  const auto st = static_cast<hipStream_t>(stream);
  bool ok;
  if (dtype == PARARNN_BF16)
    ok = act == PARARNN_BLOCK_SILU ? forward<bf16, PARARNN_BLOCK_SILU>(p, st) : forward<bf16, PARARNN_BLOCK_GELU>(p, st);
  else
    ok = act == PARARNN_BLOCK_SILU ? forward<float, PARARNN_BLOCK_SILU>(p, st) : forward<float, PARARNN_BLOCK_GELU>(p, st);
  return ok ? launched() : PARARNN_ERR_UNSUPPORTED;
}

extern "C" pararnn_status pararnn_block_gated_linear_vjp(int dtype, int act, int64_t R, int64_t D, int64_t F, const void* x,
                                                         int64_t x_stride, const void* w_gate, int64_t gate_stride, const void* w_up,
                                                         int64_t up_stride, const float* pre, const void* dh, int64_t dh_stride,
                                                         void* d_x, int64_t d_x_stride, void* d_w_gate, int64_t d_gate_stride,
                                                         void* d_w_up, int64_t d_up_stride, void* ws, size_t ws_bytes, void* stream) {
  if (!dtype_ok(dtype) || (act != PARARNN_BLOCK_SILU && act != PARARNN_BLOCK_GELU) || !sizes_ok(R, D, F))
    return PARARNN_ERR_INVALID_ARG;
  const size_t e = dtype_size(dtype);
  if (!ptr_ok(x, e, R > 0 && D > 0) || !ptr_ok(w_gate, e, F > 0 && D > 0) || !ptr_ok(w_up, e, F > 0 && D > 0) ||
      !ptr_ok(pre, 4, R > 0 && F > 0) || !ptr_ok(dh, e, R > 0 && F > 0) || !ptr_ok(d_x, e, false) || !ptr_ok(d_w_gate, e, false) ||
      !ptr_ok(d_w_up, e, false) || (d_w_gate == nullptr) != (d_w_up == nullptr) || !plane_ok(R, x_stride) ||
      !plane_ok(F, gate_stride) || !plane_ok(F, up_stride) || !plane_ok(R, dh_stride) || !plane_ok(R, d_x_stride) ||
      !plane_ok(F, d_gate_stride) || !plane_ok(F, d_up_stride))
    return PARARNN_ERR_INVALID_ARG;
  if (R > kMost || D > kMost || F > kMost) return PARARNN_ERR_UNSUPPORTED;
  if (!ws_ok(ws, ws_bytes, pararnn_block_gated_linear_workspace_bytes(dtype, R, D, F, 1))) return PARARNN_ERR_WORKSPACE;
  if (!d_x && !d_w_gate) return PARARNN_OK;
  const auto st = static_cast<hipStream_t>(stream);
  const auto run = [&](auto t, auto a) {
    using T = decltype(t);
    return backward<T, decltype(a)::value>(R, D, F, x, x_stride, w_gate, gate_stride, w_up, up_stride, pre, dh, dh_stride, d_x,
                                           d_x_stride, d_w_gate, d_gate_stride, d_w_up, d_up_stride, static_cast<T*>(ws), st);
  };
  using Silu = std::integral_constant<int, PARARNN_BLOCK_SILU>;
  using Gelu = std::integral_constant<int, PARARNN_BLOCK_GELU>;
  if (dtype == PARARNN_BF16) return act == PARARNN_BLOCK_SILU ? run(bf16{}, Silu{}) : run(bf16{}, Gelu{});
  return act == PARARNN_BLOCK_SILU ? run(0.0f, Silu{}) : run(0.0f, Gelu{});
}
