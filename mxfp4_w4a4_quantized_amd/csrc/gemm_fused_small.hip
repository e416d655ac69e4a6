// Small-M MXFP4 GEMMs with a feed-forward epilogue, and their gated form, for
// gfx950:
//   Y = residual + gate[g] * act(A B^T + bias)
//   H = act(A G^T + bias) * (A U^T + bias_u)
// dense, or requantized to MXFP4 along N after an optional Hadamard-32.
//
// The time is the weight stream, as in gemm_small.hip, whose design this
// follows (same operand addressing, K split and sums): one workgroup per 16 PG
// output columns, its waves split K, and an LDS reduction joins their partial
// tiles.  The gated form holds the matching rows of G and U in the same
// workgroup (weight fragments 0 .. PG-1 from G, PG .. 2 PG-1 from U), so both
// weights stream through one launch, the activations are read once, and the
// product is formed from the fp32 sums.  The epilogue runs on the wave that
// sums a fragment: a lane holds four consecutive columns of one row.
//
// Measured (tiled weights from HBM): 16 x 4096 -> 2 x 14336, gated silu, 62.9 MB
// in 14.2 us, 4.4 TB/s; 1 x 14336 -> 4096 with a residual, 31.2 MB in 9.6 us,
// 3.2 TB/s (start, join of the K split and end: 3 to 4 us over the bytes alone).
#include "gemm_small_core.h"
#include "activation.h"

#include <type_traits>

namespace mxfp4 {
namespace {

using namespace smallm;

// Tiled operands: the scale bytes of one K step of a 16-row fragment are 64
// contiguous bytes (row-major [16][4]).  Lane (r, g) loads the dword of row r
// for step s0 + 4 i + g, i.e. the scales of all four blocks of that step; the
// scale of step s0 + 4 i + j for the lane's own block g then sits in byte g of
// lane (r, j)'s dword.  One dword load replaces four byte loads.  Steps past
// `last` read its dword (never used).
template <int NCH>
__device__ __forceinline__ void chunk_scales(const Operand& o, int s0, int last, int lane, int (&sc)[NCH]) {
  const int lr = lane & 15, lg = lane >> 4;
#pragma unroll
  for (int i = 0; i < NCH / 4; ++i) {
    const int dw = *reinterpret_cast<const int*>(o.scale_row + (int64_t)min(s0 + 4 * i + lg, last) * o.sstride);
#pragma unroll
    for (int j = 0; j < 4; ++j) sc[4 * i + j] = __shfl(dw, 16 * j + lr) >> (8 * lg);
  }
}

// One chunk of NCH steps from s0 on into the accumulator tiles.  FULL: every
// step lies inside the wave's range and inside K; the loads have no predicates
// and constant offsets.  Otherwise steps from s_end on are left out: tiled
// operands (no K tail inside a step) load the last step again in their place,
// row-major ones take predicated loads, which also cover blocks past K.
template <int MG, int NG, bool TILED, int NCH, bool FULL>
__device__ __forceinline__ void k_chunk(const Operand (&w)[NG], const Operand (&x)[MG], v4f (&acc)[NG][MG], int s0,
                                        int s_end, int kblocks, int lane) {
  const int lg = lane >> 4;
  const int last = s_end - 1;
  auto load = [&](const Operand& o, int j, auto stream, u32x4& code, int& scale) {
    const int s = TILED && !FULL ? min(s0 + j, last) : s0 + j;
    if (FULL || TILED || (s < s_end && 4 * s + lg < kblocks)) {
      const u32x4* p = reinterpret_cast<const u32x4*>(o.code + s * o.cstride);
      if constexpr (decltype(stream)::value) code = __builtin_nontemporal_load(p);
      else code = *p;
      if constexpr (!TILED) scale = o.scale[s * o.sstride];
    } else {
      code = u32x4{0u, 0u, 0u, 0u};
      scale = 0;
    }
  };
  u32x4 wf[NG][NCH];
  int ws[NG][NCH];
#pragma unroll
  for (int j = 0; j < NCH; ++j)
#pragma unroll
    for (int q = 0; q < NG; ++q) load(w[q], j, std::true_type{}, wf[q][j], ws[q][j]);
  if constexpr (TILED) {
#pragma unroll
    for (int q = 0; q < NG; ++q) chunk_scales<NCH>(w[q], s0, last, lane, ws[q]);
  }
  // the next M group's activations load while this one's MFMAs run (not with
  // 4 x 4 accumulator tiles: no registers for it)
  constexpr int NB = MG * NG < 16 ? 2 : 1;
  u32x4 xf[NB][NCH];
  int xs[NB][NCH];
  auto load_x = [&](int mg) {
#pragma unroll
    for (int j = 0; j < NCH; ++j) load(x[mg], j, std::false_type{}, xf[mg % NB][j], xs[mg % NB][j]);
    if constexpr (TILED) chunk_scales<NCH>(x[mg], s0, last, lane, xs[mg % NB]);
  };
  load_x(0);
#pragma unroll
  for (int mg = 0; mg < MG; ++mg) {
    if (NB == 2 ? mg + 1 < MG : mg > 0) load_x(NB == 2 ? mg + 1 : mg);
    // in this order: left to itself the compiler moves the next group's loads
    // behind these MFMAs (64 rows x 4096 -> 2 x 14336: 20.9 instead of 19.5 us)
    if constexpr (MG > 1) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < NCH; ++j)
      if (FULL || s0 + j < s_end) {
#pragma unroll
        for (int q = 0; q < NG; ++q) acc[q][mg] = mma(wf[q][j], xf[mg % NB][j], acc[q][mg], ws[q][j], xs[mg % NB][j]);
      }
  }
}

// One wave's K range [s_begin, s_end): NG weight fragments against MG
// activation fragments per step, the steps in ascending order whatever the
// chunk length NCH, so that every kernel that takes the same split forms the
// same sums.
template <int MG, int NG, bool TILED, int NCH>
__device__ __forceinline__ void k_loop(const Operand (&w)[NG], const Operand (&x)[MG], v4f (&acc)[NG][MG], int s_begin,
                                       int s_end, int kblocks, int lane) {
  int s0 = s_begin;
  for (; s0 + NCH <= s_end && (TILED || 4 * (s0 + NCH) <= kblocks); s0 += NCH)
    k_chunk<MG, NG, TILED, NCH, true>(w, x, acc, s0, s_end, kblocks, lane);
  for (; s0 < s_end; s0 += NCH) k_chunk<MG, NG, TILED, NCH, false>(w, x, acc, s0, s_end, kblocks, lane);
}

// Four elements from index i on, of which the first `left` are in range (the
// others repeat the last one: no predicates).
__device__ __forceinline__ v4f load4(const void* p, bool bf16, int64_t i, int left) {
  v4f v;
  if (bf16) {
    const uint16_t* q = static_cast<const uint16_t*>(p) + i;
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = __uint_as_float((uint32_t)q[min(r, left - 1)] << 16);
  } else {
    const float* q = static_cast<const float*>(p) + i;
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = q[min(r, left - 1)];
  }
  return v;
}

// What the epilogue of one lane's four columns reads.  Rows and columns past
// the end read the last ones (their results are not stored).
template <bool GLU>
struct Extra {
  v4f bias, bias_u;
};
template <>
struct Extra<false> {
  v4f bias, gate, res;
};

template <bool GLU>
__device__ __forceinline__ void load_extra(const FusedArgs& f, int m, int n, Extra<GLU>& e) {
  m = min(m, f.g.m - 1);
  n = min(n, f.g.n - 1);
  const int left = f.g.n - n;
  if (f.bias != nullptr) e.bias = load4(f.bias, f.vec_bf16, n, left);
  if constexpr (GLU) {
    if (f.bias_u != nullptr) e.bias_u = load4(f.bias_u, f.vec_bf16, n, left);
  } else {
    if (f.gate != nullptr)
      e.gate = load4(f.gate, f.vec_bf16, (int64_t)((uint32_t)m / f.group_rows) * f.ld_gate + n, left);
    if (f.residual != nullptr) e.res = load4(f.residual, f.res_bf16, (int64_t)m * f.ld_res + n, left);
  }
}

// act on every value, chosen once
template <int N>
__device__ __forceinline__ void activate(int kind, v4f (&v)[N]) {
  float x[4 * N];
#pragma unroll
  for (int i = 0; i < 4 * N; ++i) x[i] = v[i / 4][i % 4];
  switch (kind) {
    case act::RELU: act::relu(x); break;
    case act::SILU: act::silu(x); break;
    case act::GELU: act::gelu(x); break;
    case act::GELU_TANH: act::gelu_tanh(x); break;
    default: break;
  }
#pragma unroll
  for (int i = 0; i < 4 * N; ++i) v[i / 4][i % 4] = x[i];
}

// The epilogue of N fragments of a lane: v their sums (u: the up projection's).
template <bool GLU, int N>
__device__ __forceinline__ void finish(const FusedArgs& f, const Extra<GLU> (&e)[N], v4f (&v)[N], v4f (&u)[N]) {
  if (f.bias != nullptr) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += e[i].bias;
  }
  activate(f.act, v);
  if constexpr (GLU) {
    if (f.bias_u != nullptr) {
#pragma unroll
      for (int i = 0; i < N; ++i) u[i] += e[i].bias_u;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= u[i];
  } else {
    if (f.gate != nullptr) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] *= e[i].gate;
    }
    if (f.residual != nullptr) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += e[i].res;
    }
  }
}

// One butterfly between neighbouring lane groups, of X lanes, for two registers
// at once: a permlane swap, [a0 a1] [b0 b1] -> [a0 b0] [a1 b1], makes it one
// add and one subtract, and is its own inverse.
template <int X>
__device__ __forceinline__ void butterfly_lanes(float& a, float& b) {
  auto swap = [](float p, float q) {
    if constexpr (X == 16) return __builtin_amdgcn_permlane16_swap(__float_as_uint(p), __float_as_uint(q), false, false);
    else return __builtin_amdgcn_permlane32_swap(__float_as_uint(p), __float_as_uint(q), false, false);
  };
  const auto r = swap(a, b);
  const float u = __uint_as_float(r[0]), w = __uint_as_float(r[1]);
  const auto t = swap(u + w, u - w);
  a = __uint_as_float(t[0]);
  b = __uint_as_float(t[1]);
}

// Hadamard-32 of the 32-column block of each row: lane (r, g) holds columns
// 4g + j (v0) and 16 + 4g + j (v1).  Butterflies with strides 1, 2, 4, 8, 16
// and the final multiply in the quantizer's order: strides 1 and 2 run over j,
// 4 and 8 over the lane groups, 16 over v0 and v1.
__device__ __forceinline__ void hadamard_lanes(v4f& v0, v4f& v1) {
  v4f* v[2] = {&v0, &v1};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const v4f t = *v[h];
    const float a0 = t[0] + t[1], a1 = t[0] - t[1], a2 = t[2] + t[3], a3 = t[2] - t[3];
    float b[4] = {a0 + a2, a1 + a3, a0 - a2, a1 - a3};
    butterfly_lanes<16>(b[0], b[1]);
    butterfly_lanes<16>(b[2], b[3]);
    butterfly_lanes<32>(b[0], b[1]);
    butterfly_lanes<32>(b[2], b[3]);
    *v[h] = v4f{b[0], b[1], b[2], b[3]};
  }
  const float c = __uint_as_float(0x3E3504F3u);   // nearest fp32 to 1/sqrt(32)
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float s = v0[r] + v1[r], d = v0[r] - v1[r];
    v0[r] = s * c;
    v1[r] = d * c;
  }
}

// Y[m][n .. n + 3], bounds-checked against N.
template <bool BF16>
__device__ __forceinline__ void store4(const GemmArgs& g, int m, int n, const v4f& y, int y_vec) {
  if constexpr (BF16) {
    uint16_t* yp = static_cast<uint16_t*>(g.y) + (int64_t)m * g.ld_y + n;
    const uint32_t d0 = pack_bf16(y[0], y[1]), d1 = pack_bf16(y[2], y[3]);
    if (y_vec && n + 3 < g.n) {
      *reinterpret_cast<uint2*>(yp) = make_uint2(d0, d1);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < g.n) yp[r] = (uint16_t)((r < 2 ? d0 : d1) >> (16 * (r & 1)));
    }
  } else {
    float* yp = static_cast<float*>(g.y) + (int64_t)m * g.ld_y + n;
    if (y_vec && n + 3 < g.n) {
      *reinterpret_cast<float4*>(yp) = make_float4(y[0], y[1], y[2], y[3]);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < g.n) yp[r] = y[r];
    }
  }
}

// OUT: 0 fp32 Y, 1 bf16 Y, 2 MXFP4 Y (PG == 2: one 32-block of each output
// row per workgroup).  NCH: K steps per register chunk.
template <int MG, int PG, int OUT, bool TILED, bool GLU, int NCH>
__global__ __launch_bounds__(64 * MAXW) void gemm_fused_small_kernel(FusedArgs f, int spw, int y_vec) {
  constexpr int NG = GLU ? 2 * PG : PG;
  static_assert(OUT != 2 || PG == 2, "the MXFP4 output needs 32 columns per workgroup");
  __shared__ v4f red[MAXW][MG * NG][64];

  const GemmArgs& g = f.g;
  const int lane = threadIdx.x & 63, nwaves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int n0 = blockIdx.x * 16 * PG;
  const int m0 = blockIdx.y * 16 * MAXMG;
  const int nsteps = (g.k + 127) >> 7;
  const int s_begin = wave * spw;
  const int s_end = min(nsteps, s_begin + spw);

  Operand w[NG];
#pragma unroll
  for (int q = 0; q < NG; ++q) {
    const bool up = GLU && q >= PG;
    w[q] = operand<TILED>(up ? f.u_codes : g.b_codes, up ? f.u_scales : g.b_scales, n0 + 16 * (up ? q - PG : q) + lr,
                          g.n, g.k, lg);
  }
  Operand x[MG];
#pragma unroll
  for (int mg = 0; mg < MG; ++mg) x[mg] = operand<TILED>(g.a_codes, g.a_scales, m0 + 16 * mg + lr, g.m, g.k, lg);

  v4f acc[NG][MG];
#pragma unroll
  for (int q = 0; q < NG; ++q)
#pragma unroll
    for (int mg = 0; mg < MG; ++mg) acc[q][mg] = v4f{0.f, 0.f, 0.f, 0.f};

  // Output units over the waves: the two fragments of a row group's 32-block
  // (MXFP4) or one fragment.  What the epilogue of this wave's first unit reads
  // is loaded ahead of the K loop: behind it, it costs a round trip to HBM.
  constexpr int UF = OUT == 2 ? 2 : 1, NU = MG * PG / UF;
  auto unit = [&](int i, int h, int& p, int& mg) {
    p = OUT == 2 ? h : i / MG;
    mg = OUT == 2 ? i : i % MG;
  };
  Extra<GLU> e[UF];
  auto load_unit = [&](int i) {
#pragma unroll
    for (int h = 0; h < UF; ++h) {
      int p, mg;
      unit(i, h, p, mg);
      load_extra<GLU>(f, m0 + 16 * mg + lr, n0 + 16 * p + 4 * lg, e[h]);
    }
  };
  if (wave < NU) load_unit(wave);

  k_loop<MG, NG, TILED, NCH>(w, x, acc, s_begin, s_end, g.k >> 5, lane);

#pragma unroll
  for (int q = 0; q < NG; ++q)
#pragma unroll
    for (int mg = 0; mg < MG; ++mg) red[wave][q * MG + mg][lane] = acc[q][mg];
  __syncthreads();

  // the waves' partial tiles in wave order, as gemm_small_kernel sums them
  auto total = [&](int q, int mg) {
    v4f sum = red[0][q * MG + mg][lane];
    for (int w2 = 1; w2 < nwaves; ++w2) sum += red[w2][q * MG + mg][lane];
    return sum;
  };
  for (int i = wave; i < NU; i += nwaves) {
    if (i != wave) load_unit(i);
    v4f v[UF], u[UF];
    int p, mg;
#pragma unroll
    for (int h = 0; h < UF; ++h) {
      unit(i, h, p, mg);
      v[h] = total(p, mg);
      if constexpr (GLU) u[h] = total(PG + p, mg);
    }
    finish<GLU>(f, e, v, u);
    const int m = m0 + 16 * mg + lr;
    if constexpr (OUT == 2) {
      if (f.h32) hadamard_lanes(v[0], v[1]);
      store_requant(g, m, n0, v[0], v[1], lane);
    } else {
      const int n = n0 + 16 * p + 4 * lg;
      if (m < g.m) store4<OUT == 1>(g, m, n, v[0], y_vec);
    }
  }
}

// K steps per register chunk: 8, or 4 where a chunk of 8 weight and activation
// fragments beside the accumulators spills (256 registers per lane).
constexpr int chunk_steps(int mg, int ng, bool tiled) {
  const int regs = CH * (5 * ng + (mg > 1 ? 10 : 5)) + 4 * ng * mg;
  return tiled ? (mg == 1 || regs <= 180 ? CH : CH / 2) : (mg <= 2 && regs <= 130 ? CH : CH / 2);
}

// The K split over the waves: mxfp4_gemm's (a chunk of 8 steps per wave, 8
// waves at most), but 4 waves, of 4 steps each, where that gives fewer: short K
// leaves the chip with too few loads in flight (16 rows x 2048 -> 2 x 5632,
// MXFP4 output: 6.5 instead of 6.8 us; 64 rows 9.3 instead of 13.2).  It
// depends on K alone, so dense and MXFP4 outputs are made of the same sums.
void fused_split(int k, int& nwaves, int& spw) {
  wave_split(k, nwaves, spw);
  if (nwaves >= 4) return;
  const int nsteps = (k + 127) / 128;
  nwaves = nsteps < 8 ? 1 : nsteps < 16 ? nsteps / 4 : 4;
  spw = (nsteps + nwaves - 1) / nwaves;
}

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
