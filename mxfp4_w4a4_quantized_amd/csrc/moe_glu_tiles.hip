// The tile kernels of the experts' gated products.
#include "moe_large.h"

namespace mxfp4 {

hipError_t launch_moe_glu_tiles(const MoeArgs& f, bool mid, hipStream_t s) { return large::launch_moe_act<true>(f, mid, s); }

}  // namespace mxfp4
