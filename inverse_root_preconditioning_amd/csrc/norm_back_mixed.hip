// Backward kernels of norms and joins with an fp32 stream with bf16 branches.
#include "norm_launch.h"

namespace shp {

int join_backward_mixed(const JoinArgs& a, int pieces, bool keep, bool bias, uint32_t blocks, hipStream_t stream) {
  return launch_join_backward<false, true>(a, pieces, keep, bias, blocks, stream);
}

}  // namespace shp
