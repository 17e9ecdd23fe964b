// Host-side checks of the C ABI of the block operators (include/pararnn_block.h) for a sanitizer build: argument validation and
// workspace queries, driven with invalid, boundary and empty sizes that must end with the documented status before anything
// reaches the GPU.  Built with AddressSanitizer and UndefinedBehaviorSanitizer on the host code
// (tests/test_sanitize_block_cpu.py); exits nonzero on the first wrong status, and the sanitizers stop it on any invalid access or
// undefined operation.
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "pararnn_block.h"

static int g_checks = 0;

#define EXPECT(cond)                                                                 \
  do {                                                                               \
    ++g_checks;                                                                      \
    if (!(cond)) {                                                                   \
      std::fprintf(stderr, "block_abi_validation: check failed at line %d: %s\n", __LINE__, #cond); \
      return 1;                                                                      \
    }                                                                                \
  } while (0)

template <typename T> static T* fake(uintptr_t a = 1 << 20) { return reinterpret_cast<T*>(a); }
static const int64_t kMax = INT64_MAX;
static bool refused(pararnn_status s) {
  return s == PARARNN_ERR_INVALID_ARG || s == PARARNN_ERR_UNSUPPORTED || s == PARARNN_ERR_WORKSPACE;
}

int main() {
  const int64_t sizes[] = {-kMax - 1, -1, 0, 1, 2, 63, 65, 1000, (1 << 24) - 1, 1 << 28, INT32_MAX, int64_t(1) << 32, int64_t(1) << 40,
                           int64_t(1) << 59, kMax / 16, kMax - 63, kMax};
  void* small = fake<void>(1 << 24);
  const int64_t stride[3] = {0, 0, 0}, huge[3] = {kMax, kMax, kMax};

  // every combination of sizes: queries answer, calls with a workspace of 8 bytes or of none are refused, or the problem is empty
  for (int64_t B : sizes)
    for (int64_t T : sizes)
      for (int64_t D : sizes)
        for (int64_t K : {int64_t(-1), int64_t(0), int64_t(1), int64_t(4), int64_t(8), int64_t(9), kMax}) {
          (void)pararnn_block_conv_workspace_bytes(B, T, D, K);
          (void)pararnn_block_ssm_workspace_bytes(B, T, D, K, 1, 0);
          (void)pararnn_block_ssm_workspace_bytes(B, T, D, 16, K, 1);
          (void)pararnn_block_gated_linear_workspace_bytes(PARARNN_F32, B, T, D, 1);
          (void)pararnn_block_gated_linear_workspace_bytes(PARARNN_BF16, B, T, D, static_cast<int>(K > 1));
          pararnn_block_conv c;
          std::memset(&c, 0, sizeof c);
          c.dtype = PARARNN_BF16, c.silu = 1, c.B = B, c.T = T, c.D = D, c.K = K;
          c.x = fake<void>(), c.weight = fake<float>();
          pararnn_block_conv_grad g;
          std::memset(&g, 0, sizeof g);
          g.dy = fake<void>(), g.d_x = fake<void>(), g.d_weight = fake<float>();
          // (an empty problem's gradients are zeros that a kernel writes: not called here)
          const bool some = B > 0 && T > 0 && D > 0, none = B < 0 || T < 0 || D < 0 || some;
          if (none) EXPECT(refused(pararnn_block_causal_conv_vjp(&c, &g, small, 8, nullptr)));
          if (!some || K < 1 || K > 8) {
            const pararnn_status s = pararnn_block_causal_conv(&c, fake<void>(), stride, nullptr, nullptr);
            EXPECT(refused(s) || (s == PARARNN_OK && !some));
          }
          pararnn_block_ssm q;
          std::memset(&q, 0, sizeof q);
          q.dtype = PARARNN_F32, q.B = B, q.T = T, q.D = D, q.N = 16, q.G = K;
          q.x = q.delta = q.b = q.c = fake<void>(), q.A = fake<float>();
          pararnn_block_ssm_grad h;
          std::memset(&h, 0, sizeof h);
          h.carry = fake<float>(), h.dy = h.d_x = h.d_delta = h.d_b = h.d_c = fake<void>();
          if (none) EXPECT(refused(pararnn_block_selective_scan_vjp(&q, &h, small, 8, nullptr)));
          q.G = 1, q.N = K;
          if (!some || K > 32 || K < 1) {
            const pararnn_status s = pararnn_block_selective_scan(&q, fake<void>(), stride, nullptr, nullptr, small, 8, nullptr);
            EXPECT(refused(s) || (s == PARARNN_OK && !some));
          }
          EXPECT(pararnn_block_ssm_chunks(T) >= 0);
        }
  for (int64_t R : sizes)
    for (int64_t D : sizes)
      for (int64_t F : sizes) {
        if ((R && D && F) || R < 0 || D < 0 || F < 0)
          EXPECT(refused(pararnn_block_gated_linear_vjp(PARARNN_F32, 0, R, D, F, fake<void>(), 0, fake<void>(), 0, fake<void>(), 0,
                                                        fake<float>(), fake<void>(), 0, fake<void>(), 0, fake<void>(), 0,
                                                        fake<void>(), 0, small, 8, nullptr)));
        if (R <= 0 || D < 0 || F <= 0 || R > (int64_t(1) << 40) || D > (int64_t(1) << 40) || F > (int64_t(1) << 40)) {
          const pararnn_status f = pararnn_block_gated_linear(PARARNN_BF16, 1, R, D, F, fake<void>(), 0, fake<void>(), 0, fake<void>(), 0,
                                                              fake<void>(), 0, nullptr, nullptr, 0, nullptr);
          EXPECT(refused(f) || (f == PARARNN_OK && (R == 0 || F == 0)));
        }
      }
  // strides that no offset holds, offsets without sequences, optimizer sizes
  {
    pararnn_block_conv c;
    std::memset(&c, 0, sizeof c);
    c.dtype = PARARNN_BF16, c.B = 2, c.T = 3, c.D = 4, c.K = 4, c.x = fake<void>(), c.weight = fake<float>();
    EXPECT(pararnn_block_causal_conv(&c, fake<void>(), huge, nullptr, nullptr) == PARARNN_ERR_INVALID_ARG);
    c.cu_seqlens = fake<int32_t>();
    for (int64_t n : {int64_t(-1), int64_t(0), kMax / 16, kMax}) {
      c.n_seqs = n;
      EXPECT(pararnn_block_causal_conv(&c, fake<void>(), stride, nullptr, nullptr) == PARARNN_ERR_INVALID_ARG);
    }
    pararnn_block_ssm q;
    std::memset(&q, 0, sizeof q);
    q.dtype = PARARNN_F32, q.B = 2, q.T = 3, q.D = 4, q.N = 5, q.G = 1, q.x = q.delta = q.b = q.c = fake<void>(), q.A = fake<float>();
    EXPECT(refused(pararnn_block_selective_scan(&q, fake<void>(), huge, nullptr, nullptr, small, 1 << 20, nullptr)));
    q.cu_seqlens = fake<int32_t>();
    for (int64_t n : {int64_t(-1), int64_t(0), kMax / 16, kMax}) {
      q.n_seqs = n;
      EXPECT(pararnn_block_selective_scan(&q, fake<void>(), stride, nullptr, nullptr, small, 1 << 20, nullptr) == PARARNN_ERR_INVALID_ARG);
    }
    pararnn_block_adamw_args a;
    std::memset(&a, 0, sizeof a);
    a.bits = 32, a.beta1 = 0.9, a.beta2 = 0.9, a.lr = 1, a.grad_scale = 1, a.step = kMax, a.m = a.v = fake<void>();
    for (int64_t n : sizes)
      for (int64_t o : sizes) {
        const pararnn_block_adamw_tensor t{fake<void>(), fake<void>(), n, o, 0, 0};
        if (n <= 0 || o < 0 || o % 256 || n > int64_t(1) << 40)
          EXPECT(refused(pararnn_block_adamw(&a, &t, 1, nullptr)) || (n == 0 && o >= 0 && o % 256 == 0));
        if (n <= 0 || n % 256)
          EXPECT(refused(pararnn_block_adamw_moments(n, fake<void>(), fake<void>(), fake<float>(), fake<float>(), fake<void>(), fake<void>(),
                                                     nullptr)) || n == 0);
      }
  }
  std::printf("block_abi_validation: %d checks passed\n", g_checks);
  return 0;
}
