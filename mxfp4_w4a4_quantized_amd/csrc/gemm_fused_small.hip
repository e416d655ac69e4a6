// The small-M GEMMs with an epilogue (gemm_fused_small.h): launches.
#include "gemm_fused_small.h"

namespace mxfp4 {
namespace {

template <int MG, int PG, int OUT, bool GLU, bool TILED>
void launch_layout(const FusedArgs& f, hipStream_t s) {
  constexpr int NCH = chunk_steps(MG, GLU ? 2 * PG : PG, TILED);
  int nwaves, spw;
  fused_split(f.g.k, nwaves, spw);
  const size_t ybytes = f.g.y_bf16 ? 2 : 4;
  const int y_vec = (((uintptr_t)f.g.y) % (4 * ybytes) == 0) && (f.g.ld_y % 4 == 0);
  const dim3 grid((f.g.n + 16 * PG - 1) / (16 * PG), (f.g.m + 16 * MAXMG - 1) / (16 * MAXMG));
  if (NCH == CH && spw > CH / 2)
    gemm_fused_small_kernel<MG, PG, OUT, TILED, GLU, NCH><<<grid, 64 * nwaves, 0, s>>>(f, spw, y_vec);
  else
    gemm_fused_small_kernel<MG, PG, OUT, TILED, GLU, CH / 2><<<grid, 64 * nwaves, 0, s>>>(f, spw, y_vec);
}

template <int MG, int PG, int OUT, bool GLU>
void launch(const FusedArgs& f, hipStream_t s) {
  if (f.g.tiled) launch_layout<MG, PG, OUT, GLU, true>(f, s);
  else launch_layout<MG, PG, OUT, GLU, false>(f, s);
}

// PG: output column groups of 16 per workgroup for plain dense outputs
template <int MG, int PG>
void launch_mg(const FusedArgs& f, hipStream_t s) {
  if (f.glu) {
    if (f.g.q_out) launch<MG, 2, 2, true>(f, s);
    else if (f.g.y_bf16) launch<MG, 1, 1, true>(f, s);
    else launch<MG, 1, 0, true>(f, s);
  } else {
    if (f.g.q_out) launch<MG, 2, 2, false>(f, s);
    else if (f.g.y_bf16) launch<MG, PG, 1, false>(f, s);
    else launch<MG, PG, 0, false>(f, s);
  }
}

}  // namespace

hipError_t launch_fused_small(const FusedArgs& f, hipStream_t s) {
  // Up to 32 rows, two column groups share each activation fragment, unless
  // that leaves CUs without a workgroup (16 rows x 14336 -> 4096: 11.4 us with
  // 128 workgroups, 9.5 with 256).
  const bool wide = (f.g.n + 31) / 32 >= cu_count();
  switch (f.g.m > 16 * MAXMG ? MAXMG : (f.g.m + 15) / 16) {
    case 1: wide ? launch_mg<1, 2>(f, s) : launch_mg<1, 1>(f, s); break;
    case 2: wide ? launch_mg<2, 2>(f, s) : launch_mg<2, 1>(f, s); break;
    case 3: launch_mg<3, 1>(f, s); break;
    default: launch_mg<4, 1>(f, s); break;
  }
  return hipGetLastError();
}

}  // namespace mxfp4
