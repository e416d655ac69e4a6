// The experts' products of few rows per expert (gemm_fused_small.h): row tiles of
// 16 or 32 rows, a workgroup per tile and 16 or 32 output columns.
#include "gemm_fused_small.h"

namespace mxfp4 {
namespace {

template <int MG, int PG, int OUT, bool GLU, bool TILED>
void launch_layout(const MoeArgs& f, hipStream_t s) {
  constexpr int NCH = chunk_steps(MG, GLU ? 2 * PG : PG, TILED);
  int nwaves, spw;
  fused_split(f.g.k, nwaves, spw);
  const size_t ybytes = f.g.y_bf16 ? 2 : 4;
  const int y_vec = (((uintptr_t)f.g.y) % (4 * ybytes) == 0) && (f.g.ld_y % 4 == 0);
  const int64_t tiles = moe::max_tiles(f.g.m, f.experts, 16 * MG), gy = tiles < 65535 ? tiles : 65535;
  const dim3 grid((f.g.n + 16 * PG - 1) / (16 * PG), (unsigned)gy, (unsigned)((tiles + gy - 1) / gy));
  if (NCH == CH && spw > CH / 2)
    gemm_fused_small_kernel<MG, PG, OUT, TILED, GLU, NCH><<<grid, 64 * nwaves, 0, s>>>(f, spw, y_vec);
  else
    gemm_fused_small_kernel<MG, PG, OUT, TILED, GLU, CH / 2><<<grid, 64 * nwaves, 0, s>>>(f, spw, y_vec);
}

template <int MG, int PG, int OUT, bool GLU>
void launch(const MoeArgs& f, hipStream_t s) {
  if (f.g.tiled) launch_layout<MG, PG, OUT, GLU, true>(f, s);
  else launch_layout<MG, PG, OUT, GLU, false>(f, s);
}

template <int MG>
void launch_mg(const MoeArgs& f, hipStream_t s) {
  // Two column groups of 16 share an activation fragment (512 tokens x 8 of 128
  // experts, 4096 -> 2 x 2048, row tiles of 32: 319 us with one, 259 with two).
  constexpr int PG = 2;
  if (f.glu) {
    if (f.g.q_out) launch<MG, 2, 2, true>(f, s);
    else if (f.g.y_bf16) launch<MG, PG, 1, true>(f, s);
    else launch<MG, PG, 0, true>(f, s);
  } else {
    if (f.g.q_out) launch<MG, 2, 2, false>(f, s);
    else if (f.g.y_bf16) launch<MG, PG, 1, false>(f, s);
    else launch<MG, PG, 0, false>(f, s);
  }
}

}  // namespace

hipError_t launch_moe_small(const MoeArgs& f, int rows, hipStream_t s) {
  switch (rows) {
    case 16: launch_mg<1>(f, s); break;
    default: launch_mg<2>(f, s); break;
  }
  return hipGetLastError();
}

}  // namespace mxfp4
