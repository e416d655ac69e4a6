// The large-tile GEMMs with an epilogue (gemm_fused_large.h), and the choice of
// a kernel for the GEMMs with an epilogue and their gated form.
#include "gemm_fused_large.h"

namespace mxfp4 {

// Decode shapes and shapes with fewer output tiles than XCDs take the small-M
// kernel, as mxfp4_gemm does (gemm_small_route; the gated form's tiles are 128
// columns wide).  Other shapes take the large-tile kernel where it reads the
// operands: K in whole stages, 4-byte aligned scale words and 32-bit operand
// offsets.  Row-major operands outside that stay on the small-M kernel (one
// grid row per 64 rows).
FusedRoute fused_route(const FusedArgs& f) {
  const GemmArgs& g = f.g;
  if (gemm_small_route(g.m, f.glu ? 2 * int64_t(g.n) : g.n)) return FusedRoute::kSmall;
  GemmArgs u = g;
  u.b_codes = f.u_codes;
  u.b_scales = f.u_scales;
  if (gemm_large_supported(g) && (!f.glu || gemm_large_supported(u))) return FusedRoute::kLarge;
  return g.tiled || (g.m + 63) / 64 > 65535 ? FusedRoute::kNone : FusedRoute::kSmall;
}

hipError_t launch_fused_large(const FusedArgs& f, hipStream_t s) {
  if (f.glu) return launch_glu_large(f, s);
  if (f.gate != nullptr || f.residual != nullptr) return launch_residual_large(f, s);
  return large::launch_large_act<false, false>(f, s);
}

}  // namespace mxfp4
