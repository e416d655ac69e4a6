// Launches of the tile kernels (gemm_fused_large.h) as experts' products.
#pragma once
#include "gemm_fused_large.h"

namespace mxfp4 {
namespace large {

template <class T, int ACT, int OUT, bool GLU>
hipError_t launch_moe_tile(const MoeArgs& f, hipStream_t s) {
  constexpr int TN = GLU ? T::BN / 2 : T::BN;
  const int tiles_n = (f.g.n + TN - 1) / TN;
  const int64_t most = moe::max_tiles(f.g.m, f.experts, T::BM) * tiles_n, wgs = (int64_t)cu_count() * T::WGS;
  const int grid = (int)(most < wgs ? most : wgs);
  gemm_fused_large_kernel<T, ACT, OUT, 0, GLU><<<grid, T::NT, 0, s>>>(f, 0, tiles_n, grid, 0);
  return hipGetLastError();
}

typedef Tile<128, 128, 4, 2, true> MidTail;

template <int ACT, int OUT, bool GLU>
hipError_t launch_moe(const MoeArgs& f, bool mid, hipStream_t s) {
  if (f.g.k % KS != 0) return launch_moe_tile<MidTail, ACT, OUT, GLU>(f, s);
  return mid ? launch_moe_tile<Mid, ACT, OUT, GLU>(f, s) : launch_moe_tile<Large, ACT, OUT, GLU>(f, s);
}

template <int ACT, bool GLU>
hipError_t launch_moe_out(const MoeArgs& f, bool mid, hipStream_t s) {
  if (f.g.q_out) return launch_moe<ACT, 2, GLU>(f, mid, s);
  return f.g.y_bf16 ? launch_moe<ACT, 1, GLU>(f, mid, s) : launch_moe<ACT, 0, GLU>(f, mid, s);
}

template <bool GLU>
hipError_t launch_moe_act(const MoeArgs& f, bool mid, hipStream_t s) {
  switch (f.act) {
    case act::SILU: return launch_moe_out<act::SILU, GLU>(f, mid, s);
    case act::GELU: return launch_moe_out<act::GELU, GLU>(f, mid, s);
    case act::GELU_TANH: return launch_moe_out<act::GELU_TANH, GLU>(f, mid, s);
    default: return launch_moe_out<A_LINEAR, GLU>(f, mid, s);
  }
}

}  // namespace large

hipError_t launch_moe_glu_tiles(const MoeArgs& f, bool mid, hipStream_t s);

}  // namespace mxfp4
