// lm_scan.hip -- the gated linear recurrence of pararnn_lm.h and its gradients.
//
//   a_t = exp(k sig(r_t)), k = -c softplus(lam);  h_t = a_t h_{t-1} + m_t u_t,  m = sqrt(1 - a^2), u = sig(i) x

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
  const float l = w == 1.0f ? e : kLn2 * hw_log2(w) * e / (w - 1.0f);
  return fmaxf(x, 0.0f) + l;
}

// The gates of one element.  For small |log a| q = 1 - a comes first, from the Taylor series of expm1, so that
// a = 1 - q is rounded to nearest and m^2 = 1 - a^2 = q (2 - q) has full relative accuracy (1 - exp() would lose
// it all where a is near 1, which is where these recurrences live); for large |log a| a itself comes first.
struct Gate {
  float a, w, sr, si;   // decay, 1 - a^2, sig(r), sig(i)
};
DEV Gate gate(float r, float i, float k) {
  Gate g;
  g.sr = sigmoid(r);
  g.si = sigmoid(i);
  const float z = k * g.sr;
  // -expm1(z), |z| <= 1/4: the first term left out is z^6 / 5040 of the sum, 5e-8
  const float small = -z * fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.0f / 720.0f, 1.0f / 120.0f), 1.0f / 24.0f),
                                                 1.0f / 6.0f), 0.5f), 1.0f);
  const float big = hw_exp2(kLog2e * z);
  const bool far = z < -0.25f;
  const float q = far ? 1.0f - big : small;
  g.a = far ? big : 1.0f - q;
  g.w = q * (2.0f - q);
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

// one channel of one row, all steps in order
template <typename T>
__global__ __launch_bounds__(64) void k_scan_serial(const ScanArgs p) {
  const int64_t d = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x, b = blockIdx.y;
  if (d >= p.D) return;
  const float k = -p.c * softplus(p.lam[d]);
  const T* x = static_cast<const T*>(p.x) + b * p.sx[0] + d;
  const T* r = static_cast<const T*>(p.r) + b * p.sr[0] + d;
  const T* i = static_cast<const T*>(p.i) + b * p.si[0] + d;
  T* out = static_cast<T*>(p.h) + b * p.sh[0] + d;
  const int64_t state = b * p.n * p.D + d, chunks = (p.T + CT - 1) / CT;
  int64_t t = 0;
  for (int32_t j = 0; j < p.n; ++j) {
    float h = p.h0 ? p.h0[state + j * p.D] : 0.0f;
    int64_t end = j + 1 < p.n ? p.cu[j + 1] : p.T;
    if (end > p.T) end = p.T;
    for (; t < end; ++t) {
      if (p.carry && t % CT == 0) p.carry[(b * chunks + t / CT) * p.D + d] = h;
      const Gate g = gate(to_f32(r[t * p.sr[1]]), to_f32(i[t * p.si[1]]), k);
      h = fmaf(g.a, h, root(g.w) * (g.si * to_f32(x[t * p.sx[1]])));
      out[t * p.sh[1]] = from_f32<T>(h);
    }
    if (p.h_last) p.h_last[state + j * p.D] = h;
  }
}

// the gradients of one channel of one row: chunk by chunk from the end, h rebuilt into the chunk's workspace
// rows [B][CT][D] first
template <typename T>
__global__ __launch_bounds__(64) void k_scan_grad_serial(const GradArgs p, float* rows) {
  const ScanArgs& f = p.f;
  const int64_t d = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x, b = blockIdx.y;
  if (d >= f.D) return;
  const float k = -f.c * softplus(f.lam[d]);
  const T* x = static_cast<const T*>(f.x) + b * f.sx[0] + d;
  const T* r = static_cast<const T*>(f.r) + b * f.sr[0] + d;
  const T* i = static_cast<const T*>(f.i) + b * f.si[0] + d;
  const T* dh = static_cast<const T*>(p.dh) + b * p.sdh[0] + d;
  T* dx = static_cast<T*>(p.dx) + b * p.sdx[0] + d;
  T* dr = static_cast<T*>(p.dr) + b * p.sdr[0] + d;
  T* di = static_cast<T*>(p.di) + b * p.sdi[0] + d;
  const int64_t state = b * f.n * f.D + d, chunks = (f.T + CT - 1) / CT;
  float* row = rows + b * CT * f.D + d;
  int32_t j = f.n;               // sequences j .. n-1 have been entered from their end
  float mu = 0.0f;               // gradient that reaches the state after step t
  for (int64_t ch = chunks - 1; ch >= 0; --ch) {
    const int64_t t0 = ch * CT, t1 = t0 + CT < f.T ? t0 + CT : f.T;
    float h = f.carry[(b * chunks + ch) * f.D + d], sum = 0.0f;
    int32_t s = f.cu ? sequence_of(f.cu, f.n, t0) : 0;
    for (int64_t t = t0; t < t1; ++t) {
      if (t > t0)
        while (s + 1 < f.n && f.cu[s + 1] <= t) h = f.h0 ? f.h0[state + ++s * f.D] : (++s, 0.0f);
      row[(t - t0) * f.D] = h;
      const Gate g = gate(to_f32(r[t * f.sr[1]]), to_f32(i[t * f.si[1]]), k);
      h = fmaf(g.a, h, root(g.w) * (g.si * to_f32(x[t * f.sx[1]])));
    }
    for (int64_t t = t1 - 1; t >= t0; --t) {
      // every sequence that begins after t has ended: their states' gradients are out, and the next one enters
      while (j > 0 && (j == f.n ? f.T : static_cast<int64_t>(f.cu[j])) > t) {
        if (j < f.n && p.d_h0) p.d_h0[state + j * f.D] = mu;
        --j;
        mu = p.d_last ? p.d_last[state + j * f.D] : 0.0f;
      }
      const float l = to_f32(dh[t * p.sdh[1]]) + mu, xv = to_f32(x[t * f.sx[1]]);
      const Gate g = gate(to_f32(r[t * f.sr[1]]), to_f32(i[t * f.si[1]]), k);
      const float m = root(g.w), u = g.si * xv, im = g.w > 0.0f ? hw_rcp(m) : 0.0f;
      const float e = l * (g.a * row[(t - t0) * f.D] - u * (g.a * g.a * im));
      sum = fmaf(e, g.sr, sum);
      dr[t * p.sdr[1]] = from_f32<T>(e * k * (g.sr * (1.0f - g.sr)));
      di[t * p.sdi[1]] = from_f32<T>(l * m * (u * (1.0f - g.si)));
      dx[t * p.sdx[1]] = from_f32<T>(l * m * g.si);
      mu = g.a * l;
    }
    if (p.part) p.part[(b * chunks + ch) * f.D + d] = sum;
  }
  if (p.d_h0) {
    // the first sequence with a step, then the empty ones before it (all of them, when T = 0)
    for (; j >= 0; --j) {
      if (j < f.n) p.d_h0[state + j * f.D] = mu;
      if (j > 0) mu = p.d_last ? p.d_last[state + (j - 1) * f.D] : 0.0f;
    }
  }
}

// d_lam = -c sig(lam) times the sum of the chunks' parts, rows in ascending order
__global__ __launch_bounds__(64) void k_scan_dlam(const float* part, int64_t rows, int64_t D, const float* lam, float c,
                                                  float* d_lam) {
  const int64_t d = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
  if (d >= D) return;
  float s = 0.0f;
  for (int64_t n = 0; n < rows; ++n) s += part[n * D + d];
  d_lam[d] = -c * sigmoid(lam[d]) * s;
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
  if (p->B == 0 || p->D == 0) return PARARNN_OK;
  if (!ptr_ok(p->lam, 4)) return PARARNN_ERR_INVALID_ARG;
  const size_t es = dtype_size(p->dtype);
  if (p->T > 0 && (!ptr_ok(p->x, es) || !ptr_ok(p->r, es) || !ptr_ok(p->i, es))) return PARARNN_ERR_INVALID_ARG;
  const int64_t* s[3] = {p->sx, p->sr, p->si};
  for (const int64_t* q : s)
    if (!plane_ok(p->B, q[0]) || !plane_ok(p->T, q[1])) return PARARNN_ERR_INVALID_ARG;
  if (p->B > 65535) return PARARNN_ERR_UNSUPPORTED;
  return PARARNN_OK;
}

static ScanArgs scan_args(const pararnn_lm_scan* p) {
  ScanArgs a{};
  a.x = p->x; a.r = p->r; a.i = p->i;
  for (int k = 0; k < 2; ++k) { a.sx[k] = p->sx[k]; a.sr[k] = p->sr[k]; a.si[k] = p->si[k]; }
  a.lam = p->lam; a.h0 = p->h0; a.cu = p->cu_seqlens;
  a.n = p->cu_seqlens ? static_cast<int32_t>(p->n_seqs) : 1;
  a.c = p->c; a.B = p->B; a.T = p->T; a.D = p->D;
  return a;
}

}  // namespace lm

using namespace lm;

extern "C" int64_t pararnn_lm_scan_chunks(int64_t T) { return T <= 0 ? 0 : ceil_div(T, CT); }

extern "C" size_t pararnn_lm_scan_workspace_bytes(int64_t B, int64_t T, int64_t D) {
  if (!sizes_fit(B, T, D) || !sizes_fit(B, D, CT)) return 0;
  return static_cast<size_t>(B * D * (pararnn_lm_scan_chunks(T) + CT)) * 4 + 256;
}

extern "C" pararnn_status pararnn_lm_gated_scan(const pararnn_lm_scan* prob, void* h, const int64_t sh[2], float* h_last,
                                                float* carry, void* ws, size_t ws_bytes, void* stream) {
  if (const pararnn_status st = check_scan(prob)) return st;
  if (!sh || !ptr_ok(h_last, 4, false) || !ptr_ok(carry, 4, false)) return PARARNN_ERR_INVALID_ARG;
  if (prob->B == 0 || prob->D == 0) return PARARNN_OK;
  if (prob->T > 0 && (!ptr_ok(h, dtype_size(prob->dtype)) || !plane_ok(prob->B, sh[0]) || !plane_ok(prob->T, sh[1])))
    return PARARNN_ERR_INVALID_ARG;
  if (!ptr_ok(ws, 256) || ws_bytes < pararnn_lm_scan_workspace_bytes(prob->B, prob->T, prob->D)) return PARARNN_ERR_WORKSPACE;
  ScanArgs a = scan_args(prob);
  a.h = h; a.sh[0] = sh[0]; a.sh[1] = sh[1]; a.h_last = h_last; a.carry = carry;
  const dim3 grid(static_cast<unsigned>(ceil_div(a.D, 64)), static_cast<unsigned>(a.B));
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (prob->dtype == PARARNN_BF16) k_scan_serial<bf16><<<grid, 64, 0, st>>>(a);
  else k_scan_serial<float><<<grid, 64, 0, st>>>(a);
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
  if (!ptr_ok(ws, 256) || ws_bytes < pararnn_lm_scan_workspace_bytes(prob->B, prob->T, prob->D)) return PARARNN_ERR_WORKSPACE;
  GradArgs a{};
  a.f = scan_args(prob);
  a.f.carry = const_cast<float*>(gr->carry);
  a.dh = gr->dh; a.d_last = gr->d_last; a.dx = gr->d_x; a.dr = gr->d_r; a.di = gr->d_i; a.d_h0 = gr->d_h0;
  for (int k = 0; k < 2; ++k) {
    a.sdh[k] = gr->sdh[k]; a.sdx[k] = gr->sdx[k]; a.sdr[k] = gr->sdr[k]; a.sdi[k] = gr->sdi[k];
  }
  const int64_t rows = prob->B * pararnn_lm_scan_chunks(prob->T);
  a.part = gr->d_lam ? static_cast<float*>(ws) : nullptr;
  float* hrows = static_cast<float*>(ws) + rows * prob->D;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const unsigned gd = static_cast<unsigned>(ceil_div(prob->D, 64));
  if (prob->B > 0) {
    const dim3 grid(gd, static_cast<unsigned>(prob->B));
    if (prob->dtype == PARARNN_BF16) k_scan_grad_serial<bf16><<<grid, 64, 0, st>>>(a, hrows);
    else k_scan_grad_serial<float><<<grid, 64, 0, st>>>(a, hrows);
  }
  if (gr->d_lam) k_scan_dlam<<<gd, 64, 0, st>>>(a.part, rows, prob->D, prob->lam, prob->c, gr->d_lam);
  return launched();
}

extern "C" int pararnn_lm_abi_version(void) { return PARARNN_LM_ABI_VERSION; }
