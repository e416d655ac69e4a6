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
  if constexpr (MG == 1) {
    if (!f.g.tiled) return launch_layout<MG, PG, OUT, GLU, false>(f, s);
  }
  launch_layout<MG, PG, OUT, GLU, true>(f, s);   // (rows of 32 are for tiled operands only: moe_tile_rows)
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

// ---------------------------------------------------------------------------
// The down projection of few pairs with the sum over each token's choices, in one
// launch: a workgroup owns 16 columns of y and goes through every row tile (16
// rows) of the plan.  A wave takes a tile at a time, or, with fewer tiles than
// waves, one of `parts` runs of its K, all by itself: no barrier between tiles, so
// the weights stream without a pause.  The products stay in LDS, row by row; then
// the workgroup adds up each token's, in the order of its choices.
//
// Against products in memory and a second launch: 1 token x 2 of 8 experts, 14336 ->
// 4096 16.5 -> 14.9 us; 4 tokens 36 -> 28; 8 tokens 44 -> 37; 4 tokens x 8 of 128,
// 2048 -> 4096 26 -> 24; from 128 pairs on the same (58).

constexpr int kDownPairs = 128;
constexpr int kDownWaves = 16;
constexpr int kDownRows = 16 * kDownWaves;   // of all parts
static_assert(kDownRows >= kDownPairs, "and of all pairs");

template <bool TILED>
__global__ __launch_bounds__(64 * kDownWaves) void moe_down_small_kernel(MoeArgs f, CombineArgs c) {
  // [parts][rows][16]; with more than one part 16 tiles rows, parts * tiles <= 16
  __shared__ __attribute__((aligned(16))) v4f z[kDownRows][4];
  __shared__ int16_t expert[kDownPairs];
  const GemmArgs& g = f.g;
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int n0 = blockIdx.x * 16, nsteps = (g.k + 127) >> 7;
  constexpr int HI = moe::height_index(16);
  const int tiles = moe::uniform(f.ntiles + HI);
  const int parts = tiles == 0 ? 1 : min(max(waves / tiles, 1), nsteps);
  const int spp = (nsteps + parts - 1) / parts, ld = 16 * tiles;
  constexpr int NCH = TILED ? CH : CH / 2;   // (row-major scale bytes take more registers)
  for (int u = wave; u < tiles * parts; u += waves) {
    const int tile = u / parts, part = u - tile * parts;
    const moe::i32x4 t = moe::uniform4(f.tiles[HI] + 4 * (int64_t)tile);
    const int row = t[1] + (tile - t[3]) * 16 + lr;
    Operand w[1], x[1];
    w[0] = operand<TILED>(g.b_codes + t[0] * f.w_codes, g.b_scales + t[0] * f.w_scales, n0 + lr, g.n, g.k, lg);
    x[0] = operand<TILED>(g.a_codes, g.a_scales, min(row, t[2] - 1), f.a_rows, g.k, lg);
    v4f acc[1][1] = {{v4f{0.f, 0.f, 0.f, 0.f}}};
    k_loop<1, 1, TILED, NCH>(w, x, acc, part * spp, min(nsteps, (part + 1) * spp), g.k >> 5, lane);
    if (row < t[2]) {
      z[part * ld + row][lg] = acc[0][0];
      if (part == 0 && lg == 0) expert[row] = (int16_t)t[0];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < (int)c.tokens * 4; i += blockDim.x) {
    const int t = i >> 2, q = i & 3, n = n0 + 4 * q, left = g.n - n;
    if (left <= 0) continue;
    v4f y = {0.f, 0.f, 0.f, 0.f};
    if (c.residual != nullptr) y = load4(c.residual, c.res_bf16, t * c.ld_res + n, left);
    for (int j = 0; j < c.topk; ++j) {
      const int row = c.slot[t * c.topk + j];
      if (row < 0) continue;
      v4f v = z[row][q];
      for (int p = 1; p < parts; ++p) v += z[p * ld + row][q];
      if (f.bias != nullptr) v += load4(f.bias, f.vec_bf16, (int64_t)expert[row] * g.n + n, left);
      const float weight = c.weights[t * c.topk + j];
#pragma unroll
      for (int r = 0; r < 4; ++r) y[r] = __builtin_fmaf(weight, v[r], y[r]);
    }
    GemmArgs out = g;
    out.y = c.y;
    out.ld_y = c.ld_y;
    if (c.y_bf16) store4<true>(out, t, n, y, 0);
    else store4<false>(out, t, n, y, 0);
  }
}

}  // namespace

// Few pairs (of more, the second launch is a small part) of few rows an expert, and
// columns for most CUs or little for each workgroup to read: 4 x 4 of 32, 1024 -> 1024
// 5.5 us against 5.9 in two launches, 12 x 3 of 10, 2816 -> 2816 11.3 and 13.2, but 16 x
// 8 of 32, 2048 -> 1024 17.8 and 10.3.  (Below 2^26 columns: a grid holds less than 2^32
// threads.)
bool moe_down_small(const MoeArgs& f) {
  const int64_t rows = ((int64_t)f.g.m * f.experts + f.spread - 1) / f.spread;   // to expect (all pairs at most: kDownPairs)
  const int64_t tiles = rows < f.experts ? rows : f.experts;
  return f.g.m <= kDownPairs && f.g.n < (1 << 26) && f.g.m / f.spread <= 7 &&
         (f.g.n >= 12 * cu_count() || tiles * f.g.k <= 32768);
}

hipError_t launch_moe_down_small(const MoeArgs& f, const CombineArgs& c, hipStream_t s) {
  // one workgroup of 16 waves fits on a CU, or two of 8
  const int grid = (f.g.n + 15) / 16, threads = 64 * (grid <= cu_count() ? kDownWaves : kDownWaves / 2);
  if (f.g.tiled) moe_down_small_kernel<true><<<grid, threads, 0, s>>>(f, c);
  else moe_down_small_kernel<false><<<grid, threads, 0, s>>>(f, c);
  return hipGetLastError();
}

hipError_t launch_moe_small(const MoeArgs& f, int rows, hipStream_t s) {
  switch (rows) {
    case 16: launch_mg<1>(f, s); break;
    default: launch_mg<2>(f, s); break;
  }
  return hipGetLastError();
}

}  // namespace mxfp4
