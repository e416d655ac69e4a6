// The tile kernels of the GEMM with bias and activation (gemm_fused_large.h), and
// the choice of a kernel for the GEMMs with an epilogue and their gated form.
#include "gemm_fused_large.h"

namespace mxfp4 {

// The kernel by its expected time, in units of 0.1 us (fits of graph-timed
// launches of 100 to 3584 rows, K from 2048 to 14336, on one MI355X of 256 CUs):
//  * 256 x 256 tiles, one per CU: 12 us and 0.5 us per K stage a round of tiles;
//  * 128 x 128 tiles, two per CU: 5 us and 0.5 us per stage a round, 0.3 us per
//    stage for a last round of at most one tile per CU (523 x 14336 -> 4096:
//    40 us against 82 on 48 tiles of 256 x 256; 1024 x 4096 -> 14336, 224 of
//    the larger tiles: 37 against 33);
//  * the small-M kernel: 4 us and the weights at 2.6 TB/s for every 64 rows.
// It depends on the sizes alone, so a shape's dense and MXFP4 outputs come from
// the same kernel, of the same sums.  Decode shapes (64 rows) and row-major
// operands that the tile kernels do not read take the small-M kernel.
FusedRoute fused_route(const FusedArgs& f) {
  const GemmArgs& g = f.g;
  const bool fits = (g.m + 63) / 64 <= 65535;   // the small-M kernel's grid
  if (g.m <= 64) return FusedRoute::kSmall;
  GemmArgs u = g;
  u.b_codes = f.u_codes;
  u.b_scales = f.u_scales;
  if (!gemm_large_supported(g) || (f.glu && !gemm_large_supported(u)))
    return fits && !g.tiled ? FusedRoute::kSmall : FusedRoute::kNone;
  const int64_t cus = cu_count(), nk = g.k / large::KS, wide = f.glu ? 2 * int64_t(g.n) : g.n;
  auto tiles = [&](int64_t t) { return ((g.m + t - 1) / t) * ((wide + t - 1) / t); };
  const int64_t t256 = tiles(256), t128 = tiles(128), rest = t128 % (2 * cus);
  const int64_t c256 = (t256 + cus - 1) / cus * (5 * nk + 120);
  const int64_t c128 = t128 / (2 * cus) * (5 * nk + 50) + (rest == 0 ? 0 : (rest <= cus ? 3 * nk : 5 * nk) + 50);
  const int64_t small = 40 + (g.m + 63) / 64 * (wide * (g.k / 32) * 17 / 260000);
  if (fits && small < c128 && small < c256) return FusedRoute::kSmall;
  return c128 < c256 ? FusedRoute::kMid : FusedRoute::kLarge;
}

hipError_t launch_fused_tiles(const FusedArgs& f, bool mid, hipStream_t s) {
  if (f.glu) return launch_glu_tiles(f, mid, s);
  if (f.gate != nullptr || f.residual != nullptr) return launch_residual_tiles(f, mid, s);
  return large::launch_large_act<false, false>(f, mid, s);
}

}  // namespace mxfp4
