// The tile kernels of the experts' plain products, and the choice of a kernel.
#include "moe_large.h"

namespace mxfp4 {

// The height of the row tiles, by the mean number of rows of an expert: the pairs
// over all the experts that the router spreads them over, which on one of several
// GPUs are more than the plan's (64 tokens x 8 of 128, 16 of them here: a mean of 4,
// not of 32).
//  * Tiled operands: up to 10 rows 16, and with K of 2048 to 4096 up to 18 rows 32: the
//    weights are streamed once or nearly, at 6 to 7.5 TB/s.  us in tiles of 16, 32 and
//    128 rows, weights from HBM:
//      gated, 8 of 128 experts, 4096 -> 2 x 2048: mean 10 172, 175, 202; 12 183, 180,
//        203; 18 254, 197, 208; 24 308, 214, 213
//      gated, 6 of 64, 2048 -> 2 x 1408: mean 10 36.9, 39.7, 42.0; 12 40.9, 40.0, 43.3
//      gated, 8 of 32, 7168 -> 2 x 2048: mean 10 92.9, 94.3, 90.3; 14 109, 96, 91
//      plain, 8 of 128, 2048 -> 4096: mean 10 104, 106, 118; 12 110, 109, 119; 18 142, 116, 122
//      plain, 6 of 64, 1408 -> 2048: mean 9 26.7, 31.3, 27.1; 14 30.5, 33.0, 27.2
//      plain, 2 of 8, 14336 -> 4096: mean 10 45.8, 56.3, 58.5; 14 55.7, 57.6, 58.5
//    With K below 2048 the waves of a workgroup, a run of K each, are too few for 32
//    rows to hide their loads; above 4096 the tile kernel's stream is the faster one.
//  * Row-major ones: up to 2 rows 16 (scale bytes come one by one there): gated 8 of
//    128, 4096 -> 2 x 2048: mean 2 264, 260, 240; 4 317, 311, 279; plain 2 of 8, 14336 ->
//    4096: mean 1 53.9, 59.4, 61.1; 3 84.8, 87.5, 66.6; plain 4 of 32, 2080 -> 1440: mean
//    2 19.9, 20.2, 25.7; 5 22.7, 23.4, 26.2.
//  * Then the tile kernels, of 128 rows where k is no multiple of 128, by fused_route's
//    model of their times on the tiles to expect, half a tile more for each expert
//    than its rows fill (1024 tokens x 8 of 64 experts, 2048 -> 4096: 113 us in
//    tiles of 128, 142 in 256; 1024 x 2 of 8 experts, 14336 -> 4096: 130 and 103).
// It depends on the sizes and the layout alone, so dense and MXFP4 outputs of a shape
// come from the same sums.
int moe_tile_rows(const MoeArgs& f) {
  const GemmArgs& g = f.g;
  const int64_t mean = g.m / f.spread;
  if (mean <= (g.tiled ? 10 : 2)) return 16;
  if (g.tiled && g.k >= 2048 && g.k <= 4096 && mean <= 18) return 32;
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
