// Launches of the join's kernels: the number of waves on a row and of pieces a
// lane follow from the columns.  The backward kernels of each pair of types
// are compiled in a source file of their own.
#pragma once

#include "host.h"
#include "kernels_norm.h"

namespace shp {

// f(waves, pieces) for a row of `cols` in pieces of V: the fewest waves whose lanes
// hold 2 pieces at most up to 2 of them, 4 waves up to 4 pieces, then 8.
template <int V, class F>
int with_row_shape(uint32_t cols, F&& f) {
  const uint32_t units = (cols + kWave * V - 1) / (kWave * V);
  using std::integral_constant;
  if (units <= 1) return f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  if (units <= 2) return f(integral_constant<int, 1>{}, integral_constant<int, 2>{});
  if (units <= 4) return f(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  if (units <= 8) return f(integral_constant<int, 4>{}, integral_constant<int, 2>{});
  if (units <= 16) return f(integral_constant<int, 4>{}, integral_constant<int, 4>{});
  if constexpr (V == 8) {
    return f(integral_constant<int, 8>{}, integral_constant<int, 4>{});
  } else {
    if (units <= 32) return f(integral_constant<int, 8>{}, integral_constant<int, 4>{});
    return f(integral_constant<int, 8>{}, integral_constant<int, 8>{});
  }
}
static_assert(SHAMPOO_NORM_COLS <= 8 * kWave * 4 * 8 && SHAMPOO_NORM_COLS <= 8 * kWave * 8 * 4, "columns of a row");

template <bool SB, bool BB>
int launch_join_backward(const JoinArgs& a, bool join, bool keep, bool bias, uint32_t blocks, hipStream_t stream) {
  return with_row_shape<SB ? 8 : 4>(a.cols, [&](auto w, auto p) {
    constexpr int W = decltype(w)::value, P = decltype(p)::value;
    const dim3 grid(blocks), block(kRowThreads<W>);
    if (!join) {
      if (keep) {
        hipLaunchKernelGGL((join_backward_kernel<SB, BB, W, P, false, true, true>), grid, block, 0, stream, a);
      } else {
        hipLaunchKernelGGL((join_backward_kernel<SB, BB, W, P, false, false, true>), grid, block, 0, stream, a);
      }
    } else if (keep && bias) {
      hipLaunchKernelGGL((join_backward_kernel<SB, BB, W, P, true, true, true>), grid, block, 0, stream, a);
    } else if (keep) {
      hipLaunchKernelGGL((join_backward_kernel<SB, BB, W, P, true, true, false>), grid, block, 0, stream, a);
    } else if (bias) {
      hipLaunchKernelGGL((join_backward_kernel<SB, BB, W, P, true, false, true>), grid, block, 0, stream, a);
    } else {
      hipLaunchKernelGGL((join_backward_kernel<SB, BB, W, P, true, false, false>), grid, block, 0, stream, a);
    }
    return check_launch();
  });
}

int join_backward_bf16(const JoinArgs&, bool join, bool keep, bool bias, uint32_t blocks, hipStream_t);
int join_backward_f32(const JoinArgs&, bool join, bool keep, bool bias, uint32_t blocks, hipStream_t);
int join_backward_mixed(const JoinArgs&, bool join, bool keep, bool bias, uint32_t blocks, hipStream_t);

}  // namespace shp
