// Host-side checks of the AdamW, norm and MX4 entry points built with
// AddressSanitizer and UndefinedBehaviorSanitizer (host code only; no GPU is
// touched): workspace sizes over a grid of sizes up to the extremes of their
// types, and refusals that return before any HIP call.
#include <cstdint>
#include <cstdio>
#include <limits>

#include "shampoo.h"

static int g_fail = 0;

#define EXPECT(cond)                                                     \
  do {                                                                   \
    if (!(cond)) {                                                       \
      std::fprintf(stderr, "%s:%d: expectation failed: %s\n", __FILE__, \
                   __LINE__, #cond);                                     \
      ++g_fail;                                                          \
    }                                                                    \
  } while (0)

int main() {
  void* fake = reinterpret_cast<void*>(0x10000);  // never dereferenced on these paths
  uint8_t* fb = static_cast<uint8_t*>(fake);
  float* ff = static_cast<float*>(fake);
  const shampoo_tensor* ft = static_cast<const shampoo_tensor*>(fake);
  const shampoo_segment* fs = static_cast<const shampoo_segment*>(fake);
  const int64_t big = std::numeric_limits<int64_t>::max(), low = std::numeric_limits<int64_t>::min();
  const int64_t sizes[] = {low, -1, 0, 1, 16, 17, 64, 127, 128, 129, 8192, int64_t(1) << 24, (int64_t(1) << 24) + 1,
                           int64_t(1) << 31, (int64_t(1) << 31) + 1, big};
  for (int64_t m : sizes)
    for (int64_t n : sizes)
      for (int64_t k : sizes) {
        const size_t p = shampoo_mx4_workspace_bytes(m, n, k), l = shampoo_mx4_linear_workspace_bytes(m, n, k);
        if (m < 0 || n < 0 || k < 0) EXPECT(p == 0 && l == 0);
        EXPECT(p <= (size_t(1) << 24));
        (void)l;
        EXPECT(shampoo_mx4_product(fb, fb, fb, fb, m, n, k, 1.f, 0.f, nullptr, SHAMPOO_T_F32, big, nullptr, 0,
                                   nullptr) <= 0);
        EXPECT(shampoo_mx4_linear(fake, big, fb, fb, m, n, k, nullptr, big, SHAMPOO_T_F32, nullptr, 0, nullptr) <= 0);
      }
  for (int64_t r : sizes)
    for (int64_t c : sizes) {
      EXPECT(shampoo_mx4_quantize(nullptr, SHAMPOO_T_F32, r, c, big, fb, fb, nullptr, nullptr, nullptr) <= 0);
      EXPECT(shampoo_mx4_dequantize(fb, fb, r, c, nullptr, SHAMPOO_T_BF16, big, nullptr) <= 0);
    }
  for (int64_t n : sizes) {
    const size_t w = shampoo_grad_norm_workspace_bytes(n);
    if (n <= 0) EXPECT(w == 0);
    EXPECT(w <= 8192);
    EXPECT(shampoo_grad_norm(nullptr, fs, n, SHAMPOO_T_F32, 1.f, n == 0 ? nullptr : ff, fake, w, nullptr) ==
           SHAMPOO_EINVAL);
    EXPECT(shampoo_adamw(ft, ft, nullptr, ff, 1, fs, n, SHAMPOO_T_F32, SHAMPOO_T_F32, SHAMPOO_STATE_F32, nullptr, fake,
                         nullptr, nullptr, 1e-3, 0.9, 0.95, 1e-8, 1, 0, nullptr, nullptr) <= 0);
    EXPECT(shampoo_adamw_moments(nullptr, nullptr, nullptr, nullptr, n, nullptr, nullptr, SHAMPOO_T_F32, nullptr) <= 0);
  }
  EXPECT(shampoo_adamw(ft, ft, nullptr, ff, 1, fs, 1, SHAMPOO_T_F32, SHAMPOO_T_F32, SHAMPOO_STATE_MX8, fake, fake, fb,
                       nullptr, 1e-3, 0.9, 0.95, 1e-8, 1, ~uint64_t(0), nullptr, nullptr) == SHAMPOO_EINVAL);
  EXPECT(shampoo_adamw(ft, ft, nullptr, ff, 1, fs, 1, SHAMPOO_T_F32, SHAMPOO_T_F32, SHAMPOO_STATE_F32, fake, fake,
                       nullptr, nullptr, 1e-3, 0.9, 0.95, 1e-8, std::numeric_limits<int>::min(), 0, nullptr,
                       nullptr) == SHAMPOO_EINVAL);
  if (g_fail == 0) std::printf("operator checks passed\n");
  return g_fail == 0 ? 0 : 1;
}
