// Backward kernels of norms and joins with a bf16 stream and branch.
#include "norm_launch.h"

namespace shp {

int join_backward_bf16(const JoinArgs& a, int pieces, bool keep, bool bias, uint32_t blocks, hipStream_t stream) {
  return launch_join_backward<true, true>(a, pieces, keep, bias, blocks, stream);
}

}  // namespace shp
