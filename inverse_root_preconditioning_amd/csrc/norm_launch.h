// Launches of the join's kernels: the number of waves on a row and of pieces a
// lane follow from the columns.  The backward kernels of each pair of types
// are compiled in a source file of their own.
#pragma once

#include "host.h"
#include "kernels_norm.h"

namespace shp {

// f(waves, pieces) for a row of `cols` in pieces of V.
template <int V, class F>
int with_row_shape(uint32_t cols, F&& f) {
  const uint32_t units = (cols + kWave * V - 1) / (kWave * V);
  using std::integral_constant;
  if (units <= 1) return f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  if (units <= 2) return f(integral_constant<int, 2>{}, integral_constant<int, 1>{});
  if (units <= 4) return f(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  if (units <= 8) return f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  if (units <= 16) return f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  if constexpr (V == 8) {
    return f(integral_constant<int, 16>{}, integral_constant<int, 2>{});
  } else {
    if (units <= 32) return f(integral_constant<int, 16>{}, integral_constant<int, 2>{});
    return f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  }
}
static_assert(SHAMPOO_NORM_COLS <= 16 * kWave * 2 * 8 && SHAMPOO_NORM_COLS <= 16 * kWave * 4 * 4, "columns of a row");

template <bool SB, bool BB, bool JOIN, bool KEEP, bool BIAS>
int launch_join_backward(const JoinArgs& a, uint32_t blocks, hipStream_t stream) {
  constexpr int V = SB ? 8 : 4;
  return with_row_shape<V>(a.cols, [&](auto w, auto p) {
    constexpr int W = decltype(w)::value, P = decltype(p)::value;
    const dim3 grid(blocks), block(kBackThreads<W, JOIN && BIAS>);
    if (a.cols % V == 0) {
      hipLaunchKernelGGL((join_backward_kernel<SB, BB, W, P, JOIN, KEEP, BIAS, true>), grid, block, 0, stream, a);
    } else {
      hipLaunchKernelGGL((join_backward_kernel<SB, BB, W, P, JOIN, KEEP, BIAS, false>), grid, block, 0, stream, a);
    }
    return check_launch();
  });
}

// Without a join the sums for a bias are a few registers that any kernel has.
template <bool SB, bool BB>
int launch_join_backward(const JoinArgs& a, bool join, bool keep, bool bias, uint32_t blocks, hipStream_t stream) {
  if (!join) return keep ? launch_join_backward<SB, BB, false, true, true>(a, blocks, stream)
                         : launch_join_backward<SB, BB, false, false, true>(a, blocks, stream);
  if (bias) return keep ? launch_join_backward<SB, BB, true, true, true>(a, blocks, stream)
                        : launch_join_backward<SB, BB, true, false, true>(a, blocks, stream);
  return keep ? launch_join_backward<SB, BB, true, true, false>(a, blocks, stream)
              : launch_join_backward<SB, BB, true, false, false>(a, blocks, stream);
}

int join_backward_bf16(const JoinArgs&, bool join, bool keep, bool bias, uint32_t blocks, hipStream_t);
int join_backward_f32(const JoinArgs&, bool join, bool keep, bool bias, uint32_t blocks, hipStream_t);
int join_backward_mixed(const JoinArgs&, bool join, bool keep, bool bias, uint32_t blocks, hipStream_t);

}  // namespace shp
