// The large-tile GEMM with a gate or a residual (gemm_fused_large.h).
#include "gemm_fused_large.h"

namespace mxfp4 {

hipError_t launch_residual_large(const FusedArgs& f, hipStream_t s) { return large::launch_large_act<false, true>(f, s); }

}  // namespace mxfp4
