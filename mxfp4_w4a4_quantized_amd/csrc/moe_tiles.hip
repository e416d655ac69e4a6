// The tile kernels of the experts' plain products, and the choice of a kernel.
#include "moe_large.h"

namespace mxfp4 {

// The height of the row tiles, by the mean number of rows of an expert.
int moe_tile_rows(const MoeArgs& f) {
  const int64_t mean = f.g.m / f.experts;
  const bool tiles = f.g.k % large::KS == 0;
  if (mean <= 12) return 16;
  if (mean <= 24) return 32;
  if (mean <= 48 || !tiles) return 64;
  return mean <= 512 ? 128 : 256;
}

hipError_t launch_moe_tiles(const MoeArgs& f, bool mid, hipStream_t s) {
  if (f.glu) return launch_moe_glu_tiles(f, mid, s);
  if (f.z_half) return large::launch_moe<large::A_LINEAR, 3, false>(f, mid, s);
  return large::launch_moe_act<false>(f, mid, s);
}

}  // namespace mxfp4
