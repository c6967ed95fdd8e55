// Launches of the join's backward kernels.  Those of each pair of types are
// compiled in a source file of their own.
#pragma once

#include <algorithm>

#include "host.h"
#include "kernels_norm.h"

namespace shp {

// How a row of `cols` lies in lanes, in pieces of V: one piece a lane up to 16
// waves, then as many as it takes.
struct RowLayout {
  int pieces;  // 1, 2 or 4
  uint32_t waves;
};
inline RowLayout row_layout(int64_t cols, int V) {
  const int64_t units = (cols + kWave * V - 1) / (kWave * V);
  const int pieces = units <= kMaxWaves ? 1 : units <= 2 * kMaxWaves ? 2 : 4;
  return {pieces, (uint32_t)((units + pieces - 1) / pieces)};
}
static_assert(SHAMPOO_NORM_COLS <= kMaxWaves * kWave * 2 * 8 && SHAMPOO_NORM_COLS <= kMaxWaves * kWave * 4 * 4,
              "columns of a row");

// f(pieces); a row in pieces of 8 has 2 of them at most.
template <int V, class F>
int with_pieces(int pieces, F&& f) {
  using std::integral_constant;
  if (pieces == 1) return f(integral_constant<int, 1>{});
  if constexpr (V == 8) {
    return f(integral_constant<int, 2>{});
  } else {
    return pieces == 2 ? f(integral_constant<int, 2>{}) : f(integral_constant<int, 4>{});
  }
}

// Workgroups of the backward kernel: rows that one holds side by side, and how
// many the compute units hold.  16 waves' worth of rows, so that there are few
// partial sums: joins and norms of 2^25 bf16 elements, us with 16, 8 and 4 waves: rows of 512 66, 67, - and
// 34, 35, -; of 2048 73, 72, 78 and 37, 38, 38; 1000 rows of 2048 14, 16, - and 10, 12, -.
// (Of 4 fp32 elements a lane 20 waves fit a unit.)
struct BackGrid {
  uint32_t lanes;
  int64_t resident;
};
inline BackGrid back_grid(const RowLayout& layout, int V) {
  BackGrid g;
  g.lanes = kMaxWaves / layout.waves;
  g.resident = 256 * std::max<uint32_t>(1, (V == 4 && layout.pieces == 1 ? 20 : kMaxWaves) / (layout.waves * g.lanes));
  return g;
}

template <bool SB, bool BB, bool JOIN, bool KEEP, bool BIAS>
int launch_join_backward(const JoinArgs& a, int pieces, uint32_t blocks, hipStream_t stream) {
  constexpr int V = SB ? 8 : 4;
  const dim3 grid(blocks), block(kWave * a.waves * a.lanes);
  return with_pieces<V>(pieces, [&](auto p) {
    constexpr int P = decltype(p)::value;
    const bool whole = a.cols % V == 0;
    if (whole) {
      hipLaunchKernelGGL((join_backward_kernel<SB, BB, P, JOIN, KEEP, BIAS, true>), grid, block, 0, stream, a);
    } else {
      hipLaunchKernelGGL((join_backward_kernel<SB, BB, P, JOIN, KEEP, BIAS, false>), grid, block, 0, stream, a);
    }
    return check_launch();
  });
}

// Without a join the sums for a bias are a few registers that any kernel has.
template <bool SB, bool BB>
int launch_join_backward(const JoinArgs& a, int pieces, bool keep, bool bias, uint32_t blocks, hipStream_t stream) {
  if (a.y == nullptr) return keep ? launch_join_backward<SB, BB, false, true, true>(a, pieces, blocks, stream)
                                  : launch_join_backward<SB, BB, false, false, true>(a, pieces, blocks, stream);
  if (bias) return keep ? launch_join_backward<SB, BB, true, true, true>(a, pieces, blocks, stream)
                        : launch_join_backward<SB, BB, true, false, true>(a, pieces, blocks, stream);
  return keep ? launch_join_backward<SB, BB, true, true, false>(a, pieces, blocks, stream)
              : launch_join_backward<SB, BB, true, false, false>(a, pieces, blocks, stream);
}

int join_backward_bf16(const JoinArgs&, int pieces, bool keep, bool bias, uint32_t blocks, hipStream_t);
int join_backward_f32(const JoinArgs&, int pieces, bool keep, bool bias, uint32_t blocks, hipStream_t);
int join_backward_mixed(const JoinArgs&, int pieces, bool keep, bool bias, uint32_t blocks, hipStream_t);

}  // namespace shp
