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
#include "gemm_small_core.h"
#include "activation.h"

namespace mxfp4 {
namespace {

using namespace smallm;

__device__ __forceinline__ float elem(const void* p, bool bf16, int64_t i) {
  if (bf16) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  return static_cast<const float*>(p)[i];
}

// What the epilogue of one lane's four columns reads.
struct Extra {
  v4f bias, bias_u, gate, res;
};

template <bool GLU>
__device__ __forceinline__ void load_extra(const FusedArgs& f, int m, int n, Extra& e) {
  const bool row = m < f.g.m;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const bool ok = n + r < f.g.n;
    e.bias[r] = f.bias != nullptr && ok ? elem(f.bias, f.vec_bf16, n + r) : 0.0f;
    if constexpr (GLU) {
      e.bias_u[r] = f.bias_u != nullptr && ok ? elem(f.bias_u, f.vec_bf16, n + r) : 0.0f;
    } else {
      e.gate[r] = f.gate != nullptr && ok && row
                      ? elem(f.gate, f.vec_bf16, (int64_t)((uint32_t)m / f.group_rows) * f.ld_gate + n + r)
                      : 1.0f;
      e.res[r] = f.residual != nullptr && ok && row ? elem(f.residual, f.res_bf16, (int64_t)m * f.ld_res + n + r) : 0.0f;
    }
  }
}

template <bool GLU>
__device__ __forceinline__ v4f finish(const FusedArgs& f, const Extra& e, const v4f& v, const v4f& u) {
  v4f y;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float b = f.bias != nullptr ? v[r] + e.bias[r] : v[r];
    float a = act::any(f.act, b);
    if constexpr (GLU) {
      a *= f.bias_u != nullptr ? u[r] + e.bias_u[r] : u[r];
    } else {
      if (f.gate != nullptr) a *= e.gate[r];
      if (f.residual != nullptr) a += e.res[r];
    }
    y[r] = a;
  }
  return y;
}

// Hadamard-32 of the 32-column block of each row: lane (r, g) holds columns
// 4g + j (v0) and 16 + 4g + j (v1).  Butterflies with strides 1, 2, 4, 8, 16
// and the final multiply in the quantizer's order: strides 1 and 2 run over j,
// 4 and 8 over the lane groups (the upper lane forms u - w from its partner's
// u), 16 over v0 and v1.
__device__ __forceinline__ void hadamard_lanes(v4f& v0, v4f& v1, int lane) {
  v4f* v[2] = {&v0, &v1};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    v4f& t = *v[h];
    const float a0 = t[0] + t[1], a1 = t[0] - t[1], a2 = t[2] + t[3], a3 = t[2] - t[3];
    t = v4f{a0 + a2, a1 + a3, a0 - a2, a1 - a3};
#pragma unroll
    for (int x = 16; x <= 32; x <<= 1)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float o = __shfl_xor(t[r], x);
        t[r] = (lane & x) ? o - t[r] : t[r] + o;
      }
  }
  const float c = __uint_as_float(0x3E3504F3u);   // nearest fp32 to 1/sqrt(32)
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float s = v0[r] + v1[r], d = v0[r] - v1[r];
    v0[r] = s * c;
    v1[r] = d * c;
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
  auto output = [&](int p, int mg) {
    const v4f v = total(p, mg);
    v4f u = v;
    if constexpr (GLU) u = total(PG + p, mg);
    Extra e;
    load_extra<GLU>(f, m0 + 16 * mg + lr, n0 + 16 * p + 4 * lg, e);
    return finish<GLU>(f, e, v, u);
  };
  if constexpr (OUT == 2) {
    for (int mg = wave; mg < MG; mg += nwaves) {
      v4f h0 = output(0, mg), h1 = output(1, mg);
      if (f.h32) hadamard_lanes(h0, h1, lane);
      store_requant(g, m0 + 16 * mg + lr, n0, h0, h1, lane);
    }
  } else {
    for (int i = wave; i < MG * PG; i += nwaves) {
      const int p = i / MG, mg = i % MG;
      const v4f y = output(p, mg);
      const int m = m0 + 16 * mg + lr, n = n0 + 16 * p + 4 * lg;
      if (m >= g.m) continue;
      if constexpr (OUT == 1) {
        uint16_t* yp = static_cast<uint16_t*>(g.y) + (int64_t)m * g.ld_y + n;
        if (y_vec && n + 3 < g.n) {
          *reinterpret_cast<uint2*>(yp) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (n + r < g.n) yp[r] = (uint16_t)(pack_bf16(y[r], 0.f) & 0xFFFFu);
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
  }
}

template <int MG, int PG, int OUT, bool GLU>
void launch(const FusedArgs& f, hipStream_t s) {
  constexpr int NG = GLU ? 2 * PG : PG;
  constexpr int NCH = NG * MG > 4 && NG == 4 ? CH / 2 : CH;   // 64 weight rows and several M groups: half the chunk
  int nwaves, spw;
  wave_split(f.g.k, nwaves, spw);
  const size_t ybytes = f.g.y_bf16 ? 2 : 4;
  const int y_vec = (((uintptr_t)f.g.y) % (4 * ybytes) == 0) && (f.g.ld_y % 4 == 0);
  const dim3 grid((f.g.n + 16 * PG - 1) / (16 * PG), (f.g.m + 16 * MAXMG - 1) / (16 * MAXMG));
  if (f.g.tiled)
    gemm_fused_small_kernel<MG, PG, OUT, true, GLU, NCH><<<grid, 64 * nwaves, 0, s>>>(f, spw, y_vec);
  else
    gemm_fused_small_kernel<MG, PG, OUT, false, GLU, NCH><<<grid, 64 * nwaves, 0, s>>>(f, spw, y_vec);
}

// PG: output column groups of 16 per workgroup for dense outputs
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
  switch (f.g.m > 16 * MAXMG ? MAXMG : (f.g.m + 15) / 16) {
    case 1: launch_mg<1, 2>(f, s); break;
    case 2: launch_mg<2, 2>(f, s); break;
    case 3: launch_mg<3, 1>(f, s); break;
    default: launch_mg<4, 1>(f, s); break;
  }
  return hipGetLastError();
}

}  // namespace mxfp4
