// The tile kernels of the GEMM with a gate or a residual (gemm_fused_large.h).
#include "gemm_fused_large.h"

namespace mxfp4 {

hipError_t launch_residual_tiles(const FusedArgs& f, bool mid, hipStream_t s) {
  return large::launch_large_act<false, true>(f, mid, s);
}

}  // namespace mxfp4
