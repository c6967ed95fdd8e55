// Host-side checks of the MX8, activation, norm and join entry points built with
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

// The backward kernels' launches are in files of their own, which are not built here.
namespace shp {
struct JoinArgs;
int join_backward_bf16(const JoinArgs&, int, bool, bool, uint32_t, hipStream_t) { return SHAMPOO_EHIP; }
int join_backward_f32(const JoinArgs&, int, bool, bool, uint32_t, hipStream_t) { return SHAMPOO_EHIP; }
int join_backward_mixed(const JoinArgs&, int, bool, bool, uint32_t, hipStream_t) { return SHAMPOO_EHIP; }
}  // namespace shp

int main() {
  void* fake = reinterpret_cast<void*>(0x10000);  // never dereferenced on these paths
  uint8_t* fb = static_cast<uint8_t*>(fake);
  float* ff = static_cast<float*>(fake);
  const int64_t big = std::numeric_limits<int64_t>::max(), low = std::numeric_limits<int64_t>::min();
  const int64_t sizes[] = {low, -1, 0, 1, 5, 31, 32, 33, 2048, 16384, 16385, int64_t(1) << 29, (int64_t(1) << 29) + 1,
                           int64_t(1) << 31, (int64_t(1) << 31) + 1, big};
  for (int64_t r : sizes)
    for (int64_t c : sizes) {
      EXPECT(shampoo_mx8_quantize(nullptr, SHAMPOO_T_F32, r, c, big, fb, fb, nullptr) <= 0);
      EXPECT(shampoo_mx8_dequantize(fb, fb, r, c, nullptr, SHAMPOO_T_BF16, big, nullptr) <= 0);
      EXPECT(shampoo_activation(0, nullptr, big, nullptr, 0, r, c, SHAMPOO_T_F32, fake, big, nullptr, nullptr, nullptr,
                                nullptr, nullptr) <= 0);
      EXPECT(shampoo_activation_backward(0, nullptr, big, fake, big, nullptr, 0, nullptr, nullptr, nullptr, nullptr, 0, r,
                                         c, SHAMPOO_T_F32, fake, big, nullptr, 0, nullptr) <= 0);
      for (int64_t g : sizes) {
        shampoo_join j = {};
        j.rows = r;
        j.cols = c;
        j.ld_residual = big;
        j.branch = fake;
        j.ld_branch = big;
        j.scale = 1.0;
        j.before.kind = SHAMPOO_NORM_LAYER;
        j.before.eps = 1e-6;
        j.gate_kind = SHAMPOO_GATE_ROWS;
        j.gate = fake;
        j.gate_rows = g;
        const size_t w = shampoo_join_workspace_bytes(&j);
        if (r <= 0 || c <= 0 || g <= 0 || c > SHAMPOO_NORM_COLS) EXPECT(w == 0);
        EXPECT(shampoo_join_forward(&j, fake, big, fake, big, nullptr) <= 0);  // no residual
        shampoo_join_grads d = {};
        d.d_h = fake;
        d.ld_d_h = d.ld_d_u = big;
        d.d_u = fake;
        EXPECT(shampoo_join_backward(&j, &d, fake, 0, nullptr) <= 0);
        // the kernel's arguments are formed and the launch's stand-in refuses
        j.residual = fake;
        j.before_stats = ff;
        EXPECT(shampoo_join_backward(&j, &d, fake, std::numeric_limits<size_t>::max(), nullptr) <= 0);
      }
    }
  EXPECT(shampoo_join_forward(nullptr, fake, 1, fake, 1, nullptr) == SHAMPOO_EINVAL);
  EXPECT(shampoo_join_backward(nullptr, nullptr, fake, 1, nullptr) == SHAMPOO_EINVAL);
  if (g_fail == 0) std::printf("layer checks passed\n");
  return g_fail == 0 ? 0 : 1;
}
