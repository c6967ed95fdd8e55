// C entry points of the AdamW step and the gradient norm (gfx950): arguments
// are checked on the host, kernels enqueued on the caller's stream; nothing
// is allocated and nothing synchronises.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "kernels_adamw.h"

using namespace shp;

namespace {

// A launch has fewer than 2^32 threads along x, 256 of them in a workgroup.
constexpr int64_t kMaxGrid = 0xffffffff / 256;
constexpr int kNormBlocks = 1024;
// Up to here one workgroup does it all: beyond, one compute unit's reading
// (8 KB a segment of fp32) takes longer than a second launch.  Whole calls on
// one tensor: 32 segments 5.1 us, 64 9.5 (bf16 8.6), any number in two launches 9.0.
constexpr int64_t kNormSmall = 64;

int check_launch() { return hipGetLastError() == hipSuccess ? SHAMPOO_OK : SHAMPOO_EHIP; }

bool valid_type(int t) { return t == SHAMPOO_T_F32 || t == SHAMPOO_T_BF16; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int norm_blocks(int64_t nseg) { return (int)(nseg < kNormBlocks ? nseg : kNormBlocks); }

// The part of the hash's counter that a whole step shares.
uint32_t step_key(uint64_t seed, int step) {
  const uint32_t s = hash_finish((uint32_t)seed * kHashC1 + (uint32_t)(seed >> 32) * kHashC4);
  return hash_finish(s + (uint32_t)step * kHashC1);
}

template <bool PARAM_BF16, bool GRAD_BF16, bool MX8, bool TINY>
int launch_copy(const AdamwArgs& a, uint32_t grid, hipStream_t stream) {
  if (a.copies != nullptr) {
    if constexpr (!PARAM_BF16)
      hipLaunchKernelGGL((adamw_kernel<false, GRAD_BF16, MX8, true, TINY>), dim3(grid), dim3(256), 0, stream, a);
  } else {
    hipLaunchKernelGGL((adamw_kernel<PARAM_BF16, GRAD_BF16, MX8, false, TINY>), dim3(grid), dim3(256), 0, stream, a);
  }
  return check_launch();
}

template <bool PARAM_BF16, bool GRAD_BF16>
int launch(const AdamwArgs& a, bool mx8, uint32_t grid, hipStream_t stream) {
  // The root of a subnormal is below 2^-63: beside such an eps it is less than half an ulp.
  const bool covered = a.eps >= 0x1p-38f * a.rsbc2;
  if (covered)
    return mx8 ? launch_copy<PARAM_BF16, GRAD_BF16, true, false>(a, grid, stream)
               : launch_copy<PARAM_BF16, GRAD_BF16, false, false>(a, grid, stream);
  return mx8 ? launch_copy<PARAM_BF16, GRAD_BF16, true, true>(a, grid, stream)
             : launch_copy<PARAM_BF16, GRAD_BF16, false, true>(a, grid, stream);
}

}  // namespace

extern "C" {

size_t shampoo_grad_norm_workspace_bytes(int64_t nsegments) {
  if (nsegments <= kNormSmall) return 0;
  return (size_t)norm_blocks(nsegments) * sizeof(double);
}

int shampoo_grad_norm(const shampoo_tensor* tensors, const shampoo_segment* segments, int64_t nsegments, int dtype,
                      float max_norm, float* out, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (nsegments < 0 || !(max_norm > 0.f) || out == nullptr) return SHAMPOO_EINVAL;
  if (!valid_type(dtype)) return SHAMPOO_EUNSUPPORTED;
  if (nsegments > 0 && (tensors == nullptr || segments == nullptr)) return SHAMPOO_EINVAL;
  const bool bf16 = dtype == SHAMPOO_T_BF16;
  if (nsegments <= kNormSmall) {
    if (bf16) {
      hipLaunchKernelGGL(grad_norm_small_kernel<true>, dim3(1), dim3(1024), 0, stream, tensors, segments,
                         (int)nsegments, max_norm, out);
    } else {
      hipLaunchKernelGGL(grad_norm_small_kernel<false>, dim3(1), dim3(1024), 0, stream, tensors, segments,
                         (int)nsegments, max_norm, out);
    }
    return check_launch();
  }
  if (ws == nullptr || ws_bytes < shampoo_grad_norm_workspace_bytes(nsegments)) return SHAMPOO_EWORKSPACE;
  if ((reinterpret_cast<uintptr_t>(ws) & 7) != 0) return SHAMPOO_EINVAL;
  const int blocks = norm_blocks(nsegments);
  double* partial = static_cast<double*>(ws);
  if (bf16) {
    hipLaunchKernelGGL(grad_norm_partial_kernel<true>, dim3(blocks), dim3(256), 0, stream, tensors, segments,
                       nsegments, partial);
  } else {
    hipLaunchKernelGGL(grad_norm_partial_kernel<false>, dim3(blocks), dim3(256), 0, stream, tensors, segments,
                       nsegments, partial);
  }
  if (check_launch() != SHAMPOO_OK) return SHAMPOO_EHIP;
  hipLaunchKernelGGL(grad_norm_final_kernel, dim3(1), dim3(256), 0, stream, partial, blocks, max_norm, out);
  return check_launch();
}

int shampoo_adamw(const shampoo_tensor* params, const shampoo_tensor* grads, const shampoo_tensor* copies,
                  const float* hyper, int64_t ntensors, const shampoo_segment* segments, int64_t nsegments,
                  int param_dtype, int grad_dtype, int state, void* m, void* v, uint8_t* m_scale, uint8_t* v_scale,
                  double lr, double beta1, double beta2, double eps, int step, uint64_t seed,
                  const float* grad_scale, hipStream_t stream) {
  if (ntensors < 0 || nsegments < 0 || step < 1 || !std::isfinite(lr)) return SHAMPOO_EINVAL;
  if (!(beta1 >= 0. && beta1 < 1.) || !(beta2 >= 0. && beta2 < 1.) || !(eps >= 0.) || std::isinf(eps))
    return SHAMPOO_EINVAL;
  if (!valid_type(param_dtype) || !valid_type(grad_dtype)) return SHAMPOO_EUNSUPPORTED;
  if (state != SHAMPOO_STATE_F32 && state != SHAMPOO_STATE_MX8) return SHAMPOO_EUNSUPPORTED;
  if (copies != nullptr && param_dtype != SHAMPOO_T_F32) return SHAMPOO_EUNSUPPORTED;
  if (ntensors == 0 || nsegments == 0) return SHAMPOO_OK;
  if (params == nullptr || grads == nullptr || hyper == nullptr || segments == nullptr || m == nullptr ||
      v == nullptr)
    return SHAMPOO_EINVAL;
  const bool mx8 = state == SHAMPOO_STATE_MX8;
  if (mx8 != (m_scale != nullptr) || mx8 != (v_scale != nullptr)) return SHAMPOO_EINVAL;
  if (!aligned16(m) || !aligned16(v)) return SHAMPOO_EINVAL;
  if (nsegments > kMaxGrid) return SHAMPOO_EUNSUPPORTED;
  AdamwArgs a;
  a.params = params;
  a.grads = grads;
  a.copies = copies;
  a.hyper = hyper;
  a.segments = segments;
  a.ntensors = ntensors;
  a.m = m;
  a.v = v;
  a.m_scale = m_scale;
  a.v_scale = v_scale;
  a.grad_scale = grad_scale;
  a.lr = (float)lr;
  a.beta1 = (float)beta1;
  a.omb1 = 1.0 - beta1;
  a.beta2 = (float)beta2;
  a.omb2 = 1.0 - beta2;
  // A subnormal eps would count as 0 in the kernel's reciprocal.  FLT_MIN serves
  // as well: it vanishes beside the least root of a v > 0, 2^-74.5.
  a.eps = eps > 0. ? std::max((float)eps, FLT_MIN) : 0.f;
  a.rbc1 = (float)(1.0 / (1.0 - std::pow(beta1, step)));
  a.rsbc2 = (float)(1.0 / std::sqrt(1.0 - std::pow(beta2, step)));
  a.key = step_key(seed, step);
  const bool gb = grad_dtype == SHAMPOO_T_BF16;
  if (param_dtype == SHAMPOO_T_BF16) return gb ? launch<true, true>(a, mx8, (uint32_t)nsegments, stream)
                                               : launch<true, false>(a, mx8, (uint32_t)nsegments, stream);
  return gb ? launch<false, true>(a, mx8, (uint32_t)nsegments, stream)
            : launch<false, false>(a, mx8, (uint32_t)nsegments, stream);
}

int shampoo_adamw_moments(const uint8_t* m, const uint8_t* m_scale, const uint8_t* v, const uint8_t* v_scale,
                          int64_t n, void* m_out, void* v_out, int dtype, hipStream_t stream) {
  if (n < 0 || n % kGroup != 0) return SHAMPOO_EINVAL;
  if (!valid_type(dtype)) return SHAMPOO_EUNSUPPORTED;
  if ((m == nullptr) != (m_scale == nullptr) || (m == nullptr) != (m_out == nullptr)) return SHAMPOO_EINVAL;
  if ((v == nullptr) != (v_scale == nullptr) || (v == nullptr) != (v_out == nullptr)) return SHAMPOO_EINVAL;
  if (n == 0) return SHAMPOO_OK;
  if (m == nullptr && v == nullptr) return SHAMPOO_EINVAL;
  const int64_t blocks = (n + 2047) / 2048;
  if (blocks > kMaxGrid) return SHAMPOO_EUNSUPPORTED;
  MomentsArgs a;
  a.codes[0] = m;
  a.codes[1] = v;
  a.scales[0] = m_scale;
  a.scales[1] = v_scale;
  a.out[0] = m_out;
  a.out[1] = v_out;
  a.n = n;
  a.first = m == nullptr ? 1 : 0;
  const dim3 grid((uint32_t)blocks, m != nullptr && v != nullptr ? 2 : 1);
  if (dtype == SHAMPOO_T_BF16) {
    hipLaunchKernelGGL(mx8_decode_kernel<true>, grid, dim3(256), 0, stream, a);
  } else {
    hipLaunchKernelGGL(mx8_decode_kernel<false>, grid, dim3(256), 0, stream, a);
  }
  return check_launch();
}

}  // extern "C"
