// The tile kernels of the experts' plain products, and the choice of a kernel.
#include "moe_large.h"

namespace mxfp4 {

// The height of the row tiles, by the mean number of rows of an expert: the pairs
// over all the experts that the router spreads them over, which on one of several
// GPUs are more than the plan's (64 tokens x 8 of 128, 16 of them here: a mean of 4,
// not of 32).
//  * Up to 7 rows 16, up to 18 rows 32: the weights are streamed once or nearly, at 6
//    to 7.5 TB/s (8 of 128 experts, 4096 -> 2 x 2048, gated; us in tiles of 16, 32 and
//    128 rows: mean 6 161, 171, 193; 8 169, 166, 189; 12 199, 179, 197; 20 269, 218,
//    210).  From k = 8192 on up to 10 rows: there the tile kernel's stream is the
//    faster one (2 of 8 experts, 14336 -> 4096: mean 12 57 in 32, 43 in 128).
//  * Then the tile kernels, of 128 rows where k is no multiple of 128, by fused_route's
//    model of their times on the tiles to expect, half a tile more for each expert
//    than its rows fill (1024 tokens x 8 of 64 experts, 2048 -> 4096: 113 us in
//    tiles of 128, 142 in 256; 1024 x 2 of 8 experts, 14336 -> 4096: 130 and 103).
// It depends on the sizes alone, so dense and MXFP4 outputs of a shape come from the
// same sums.
int moe_tile_rows(const MoeArgs& f) {
  const GemmArgs& g = f.g;
  const int64_t mean = g.m / f.spread;
  if (mean <= 7) return 16;
  if (mean <= (g.k >= 8192 ? 10 : 18)) return 32;
  if (g.k % large::KS != 0) return 128;
  const int64_t rows = (int64_t)g.m * f.experts / f.spread;   // to expect
  const int64_t cus = cu_count(), nk = g.k / large::KS, wide = f.glu ? 2 * int64_t(g.n) : g.n;
  auto tiles = [&](int64_t t) { return (rows / t + (f.experts + 1) / 2) * ((wide + t - 1) / t); };
  const int64_t t256 = tiles(256), t128 = tiles(128), rest = t128 % (2 * cus);
  const int64_t c256 = (t256 + cus - 1) / cus * (5 * nk + 120);
  const int64_t c128 = t128 / (2 * cus) * (5 * nk + 50) + (rest == 0 ? 0 : (rest <= cus ? 3 * nk : 5 * nk) + 50);
  return c128 < c256 ? 128 : 256;
}

hipError_t launch_moe_tiles(const MoeArgs& f, bool mid, hipStream_t s) {
  if (f.glu) return launch_moe_glu_tiles(f, mid, s);
  if (f.z_half) return large::launch_moe<large::A_LINEAR, 3, false>(f, mid, s);
  return large::launch_moe_act<false>(f, mid, s);
}

}  // namespace mxfp4
