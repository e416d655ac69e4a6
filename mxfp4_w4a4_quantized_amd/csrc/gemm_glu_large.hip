// The tile kernels of the gated GEMM (gemm_fused_large.h).
#include "gemm_fused_large.h"

namespace mxfp4 {

hipError_t launch_glu_tiles(const FusedArgs& f, bool mid, hipStream_t s) {
  return large::launch_large_act<true, false>(f, mid, s);
}

}  // namespace mxfp4
