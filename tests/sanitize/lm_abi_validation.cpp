// Host-side checks of the C ABI of the language-model operators (include/pararnn_lm.h) for a sanitizer build: argument
// validation and workspace queries, driven with invalid, boundary and empty sizes that must end with the documented status
// before anything reaches the GPU.  Built with AddressSanitizer and UndefinedBehaviorSanitizer on the host code
// (tests/test_sanitize_cpu.py); exits nonzero on the first wrong status, and the sanitizers stop it on any invalid access or
// undefined operation.
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "pararnn_lm.h"

static int g_checks = 0;

#define EXPECT(cond)                                                                 \
  do {                                                                               \
    ++g_checks;                                                                      \
    if (!(cond)) {                                                                   \
      std::fprintf(stderr, "lm_abi_validation: check failed at line %d: %s\n", __LINE__, #cond); \
      return 1;                                                                      \
    }                                                                                \
  } while (0)

template <typename T> static T* fake(uintptr_t a = 1 << 20) { return reinterpret_cast<T*>(a); }

static const int64_t kMax = INT64_MAX;
// statuses that a call may have without touching the GPU
static bool refused(pararnn_status s) {
  return s == PARARNN_ERR_INVALID_ARG || s == PARARNN_ERR_UNSUPPORTED || s == PARARNN_ERR_WORKSPACE;
}

static pararnn_lm_scan scan(int64_t B, int64_t T, int64_t D, int64_t n = 0, int64_t stride = 0) {
  pararnn_lm_scan p;
  std::memset(&p, 0, sizeof p);
  p.dtype = PARARNN_BF16;
  p.c = 8.0f;
  p.B = B; p.T = T; p.D = D;
  p.x = p.r = p.i = fake<void>();
  for (int k = 0; k < 2; ++k) p.sx[k] = p.sr[k] = p.si[k] = stride;
  p.lam = fake<float>();
  if (n) p.cu_seqlens = fake<int32_t>(), p.n_seqs = n;
  return p;
}

static pararnn_lm_scan_grad grad(int64_t stride = 0) {
  pararnn_lm_scan_grad g;
  std::memset(&g, 0, sizeof g);
  g.carry = fake<float>();
  g.dh = fake<void>();
  g.d_x = g.d_r = g.d_i = fake<void>();
  for (int k = 0; k < 2; ++k) g.sdh[k] = g.sdx[k] = g.sdr[k] = g.sdi[k] = stride;
  return g;
}

int main() {
  const int64_t sizes[] = {-kMax - 1, -1, 0, 1, 2, 63, 64, 65, 1000, 16384, 16385, (1 << 24) - 1, 1 << 24, (1 << 28) - 16, 1 << 28,
                           INT32_MAX, int64_t(1) << 32, int64_t(1) << 40, int64_t(1) << 59, kMax / 16, kMax - 63, kMax};
  void* ws = fake<void>(1 << 24);

  // ---- queries: any sizes ----
  for (int64_t a : sizes) {
    EXPECT(pararnn_lm_scan_chunks(a) >= 0);
    EXPECT(pararnn_lm_scan_chunks(a) == (a <= 0 ? 0 : (a - 1) / PARARNN_LM_SCAN_CHUNK + 1));
    for (int64_t b : sizes) {
      const size_t norm = pararnn_lm_layer_norm_vjp_workspace_bytes(a, b);
      EXPECT(a >= 0 && b >= 0 ? norm < SIZE_MAX / 2 : norm == 0);
      for (int top : {-1, 0, 1, 32, 33}) EXPECT(pararnn_lm_token_logprobs_workspace_bytes(a, b, top) <= 256);
      for (int64_t c : sizes) {
        const size_t n = pararnn_lm_scan_workspace_bytes(a, b, c);
        EXPECT(a >= 0 && b >= 0 && c >= 0 ? n < SIZE_MAX / 2 : n == 0);
      }
    }
  }

  // ---- the recurrence: a workspace of 16 bytes is too small for whatever passes the other checks ----
  const int64_t sh[2] = {0, 0};
  for (int64_t B : sizes)
    for (int64_t T : sizes)
      for (int64_t D : sizes)
        for (int64_t n : {int64_t(0), int64_t(1), int64_t(INT32_MAX), kMax})
          for (int64_t st : {int64_t(0), int64_t(1) << 40, kMax}) {
            const pararnn_lm_scan p = scan(B, T, D, n, st);
            const pararnn_lm_scan_grad g = grad(st);
            const bool nothing = D == 0 || B == 0;
            const pararnn_status f = pararnn_lm_gated_scan(&p, fake<void>(), sh, nullptr, nullptr, ws, 16, nullptr);
            EXPECT(refused(f) || (nothing && f == PARARNN_OK));
            const pararnn_status b = pararnn_lm_gated_scan_vjp(&p, &g, ws, 16, nullptr);
            EXPECT(refused(b) || (D == 0 && b == PARARNN_OK));
          }
  EXPECT(pararnn_lm_gated_scan(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr) == PARARNN_ERR_INVALID_ARG);
  EXPECT(pararnn_lm_gated_scan_vjp(nullptr, nullptr, nullptr, 0, nullptr) == PARARNN_ERR_INVALID_ARG);

  // ---- layer norm: a null weight, a small workspace ----
  for (int64_t N : sizes)
    for (int64_t D : sizes)
      for (int64_t st : {int64_t(-1), int64_t(0), int64_t(1) << 40, kMax}) {
        const bool nothing = N == 0 || D == 0;
        const pararnn_status f = pararnn_lm_layer_norm(PARARNN_F32, N, D, fake<void>(), st, nullptr, 0, nullptr, nullptr, 1e-5f,
                                                       fake<void>(), st, nullptr, 0, nullptr, nullptr);
        EXPECT(refused(f) || (nothing && f == PARARNN_OK));
        const pararnn_status b =
            pararnn_lm_layer_norm_vjp(PARARNN_F32, N, D, fake<void>(), st, fake<void>(), st, fake<float>(), fake<float>(), nullptr,
                                      0, fake<void>(), st, nullptr, nullptr, ws, 16, nullptr);
        EXPECT(refused(b) || (D == 0 && b == PARARNN_OK));
      }

  // ---- log probabilities: a small workspace, null statistics ----
  for (int64_t N : sizes)
    for (int64_t V : sizes)
      for (int64_t st : {int64_t(-1), int64_t(0), int64_t(1) << 40, kMax})
        for (int top : {0, 1, 32}) {
          const pararnn_status f =
              pararnn_lm_token_logprobs(PARARNN_BF16, N, V, fake<void>(), st, fake<void>(), 4, fake<float>(), fake<float>(),
                                        fake<float>(), top, fake<float>(), fake<int64_t>(), ws, 16, nullptr);
          EXPECT(refused(f) || (N == 0 && f == PARARNN_OK));
          const pararnn_status b = pararnn_lm_token_logprobs_vjp(PARARNN_BF16, N, V, fake<void>(), st, fake<void>(), 8, nullptr,
                                                                 nullptr, fake<float>(), nullptr, fake<void>(), st, nullptr);
          EXPECT(refused(b) || ((N == 0 || V == 0) && b == PARARNN_OK));
        }
  std::printf("lm_abi_validation: %d checks passed\n", g_checks);
  return 0;
}
