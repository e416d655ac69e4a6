// Shared parts of the small-M kernels (gemm_small.hip, gemm_fused_small.hip):
// operand addressing, the MXFP4 store and the K split.  The design is described
// in gemm_small.hip.
#pragma once
#include "internal.h"
#include "block_quant.h"

namespace mxfp4 {
namespace smallm {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int CH = 8;      // K steps (128 elements each) per register chunk
constexpr int MAXW = 8;    // waves per workgroup (K split)
constexpr int MAXMG = 4;   // 16-row M groups (M <= 64)
constexpr int MAXACC = 4;  // NG * MG accumulator tiles per wave

__device__ __forceinline__ int tiled_swz(int r) { return ((r >> 1) ^ (r >> 2)) & 3; }

__device__ __forceinline__ v4f mma(const u32x4& a, const u32x4& b, const v4f& c, int sa, int sb) {
  const v8i av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const v8i bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, sa, 0, sb);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  const b2 h = __builtin_convertvector(f2{a, b}, b2);
  uint32_t u;
  __builtin_memcpy(&u, &h, 4);
  return u;
}

// Operand addressing for one lane: the fragment of K step s is 16 code bytes
// at code + s * cstride and one scale byte at scale + s * sstride.
struct Operand {
  const uint8_t* code;
  const uint8_t* scale;
  int64_t cstride, sstride;
  const uint8_t* scale_row;   // tiled: the row's 4 scale bytes of stage 0
};

template <bool TILED>
__device__ __forceinline__ Operand operand(const uint8_t* codes, const uint8_t* scales, int row,
                                           int rows, int k, int lg) {
  Operand o;
  if constexpr (TILED) {
    const int64_t nstage = k >> 7;
    const int64_t t = row >> 8;
    const int r = row & 255;
    o.code = codes + t * nstage * 16384 + r * 64 + 16 * (lg ^ tiled_swz(r));
    o.scale_row = scales + t * nstage * 1024 + r * 4;
    o.scale = o.scale_row + lg;
    o.cstride = 16384;
    o.sstride = 1024;
  } else {
    const int64_t rr = row < rows ? row : rows - 1;
    o.code = codes + rr * (k >> 1) + 16 * lg;
    o.scale = scales + rr * (k >> 5) + lg;
    o.scale_row = o.scale;
    o.cstride = 64;
    o.sstride = 4;
  }
  return o;
}

// MXFP4 output of the small-M kernel: Y requantized per 32-block along N by
// the quantizer's rule, from the same fp32 sums that the fp32 output stores.
// The workgroup's 32 weight rows (NG = 2) are one block of each output row:
// lane (r, g) holds columns 4g .. 4g + 3 of fragment 0 (v0) and of fragment 1
// (v1), i.e. code bytes 2g, 2g + 1 and 8 + 2g, 8 + 2g + 1 of row r's block.
// The block amax comes from the four lanes of row r (an exact max), the codes
// from the E2M1 converter at the block scale, and lane (r, 0) gathers the 16
// code bytes and stores them with the scale byte.
__device__ __forceinline__ void store_requant(const GemmArgs& g, int m, int n0, const v4f& v0, const v4f& v1,
                                              int lane) {
  float am = 0.0f;
#pragma unroll
  for (int r = 0; r < 4; ++r) am = fmaxf(am, fmaxf(fabsf(v0[r]), fabsf(v1[r])));
  am = fmaxf(am, __shfl_xor(am, 16));
  am = fmaxf(am, __shfl_xor(am, 32));
  const uint32_t sbyte = blockq::sbyte_of_amax(am);
  const float sc = blockq::scale_of(sbyte);
  uint32_t w0 = 0, w1 = 0;
  w0 = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w0, v0[0], v0[1], sc, 0);
  w0 = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w0, v0[2], v0[3], sc, 1);
  w1 = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w1, v1[0], v1[1], sc, 0);
  w1 = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w1, v1[2], v1[3], sc, 1);
  const int lr = lane & 15;
  uint32_t p0[4], p1[4];   // the low 16 bits of w0, w1 of lanes (r, 0..3)
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    p0[j] = (uint32_t)__shfl((int)w0, lr + 16 * j) & 0xFFFFu;
    p1[j] = (uint32_t)__shfl((int)w1, lr + 16 * j) & 0xFFFFu;
  }
  if ((lane >> 4) != 0 || m >= g.m) return;
  const uint4 codes = make_uint4(p0[0] | (p0[1] << 16), p0[2] | (p0[3] << 16), p1[0] | (p1[1] << 16),
                                 p1[2] | (p1[3] << 16));
  const int blk = n0 >> 5;
  if (g.q_tiled) {
    const uint32_t r8 = (uint32_t)m & 255u, c = (uint32_t)blk & 3u;
    const uint64_t ts = (uint64_t)((uint32_t)m >> 8) * ((uint32_t)g.n >> 7) + ((uint32_t)blk >> 2);
    *reinterpret_cast<uint4*>(g.q_codes + ts * 16384 + r8 * 64 + 16 * (c ^ tiled_swz((int)r8))) = codes;
    g.q_scales[ts * 1024 + r8 * 4 + c] = (uint8_t)sbyte;
  } else {
    *reinterpret_cast<uint4*>(g.q_codes + (int64_t)m * (g.n >> 1) + 16 * blk) = codes;
    g.q_scales[(int64_t)m * (g.n >> 5) + blk] = (uint8_t)sbyte;
  }
}

// K split over the waves: chunks of CH steps, up to MAXW waves (the fused
// layer takes the same split as the small-M GEMM, so their sums agree)
inline void wave_split(int k, int& nwaves, int& spw) {
  const int nsteps = (k + 127) / 128;
  nwaves = (nsteps + CH - 1) / CH;
  if (nwaves > MAXW) nwaves = MAXW;
  if (nwaves < 1) nwaves = 1;
  spw = (nsteps + nwaves - 1) / nwaves;
}

}  // namespace smallm
}  // namespace mxfp4
