// The large-tile gated GEMM (gemm_fused_large.h).
#include "gemm_fused_large.h"

namespace mxfp4 {

hipError_t launch_glu_large(const FusedArgs& f, hipStream_t s) { return large::launch_large_act<true, false>(f, s); }

}  // namespace mxfp4
