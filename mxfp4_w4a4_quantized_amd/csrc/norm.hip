// Norm with what surrounds it in a transformer block, for gfx950:
//   p = [norm(x) * post_weight | x]
//   r = residual_scale * residual + gate[g] * p        -> residual_out
//   y = (norm(r) * weight + bias) * (1 + scale[g]) + shift[g]
// y dense, or quantized to MXFP4 after an optional block transform.
//
// Bound by HBM: x and the residual are read once, r and y (or 4.25 bits an
// element of y) written once (57344 x 3072, layer norm with gate and modulation:
// 1.41 GB in 244 us, 5.8 TB/s; a large copy reaches 5.1-5.5).  A workgroup of 1
// to 16 waves owns a row; every lane keeps its columns of the row in registers
// as chunks of 8 consecutive elements (16 bytes of bf16: a wave's load
// instruction covers 1 KiB of the row), so the statistics, which need the whole
// row, cost no second read.  Statistics are fp32: per-lane sums, then the wave's
// sum by lane permutes, then (several waves) one LDS exchange; the layer norm's
// variance is the mean square of the centred values, not a difference of moments.
//
// MXFP4 result: a 32-element block is four neighbouring lanes (a quad), so the
// block amax and the Hadamard's strides 8 and 16 are quad permutes and a lane
// stores the 4 code bytes of its chunk.  A Kronecker transform mixes all 32
// elements: there the row passes through LDS and Q lanes take a block.
// Every operation from y on is the quantizer's, in its order, so codes and
// scales equal quantizing the fp32 y bit for bit.
#include "internal.h"
#include "block_quant.h"

#include <algorithm>

namespace mxfp4 {
namespace {

using namespace blockq;

constexpr int MAXW = 16;   // waves per row at most

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, b2));
}

// Eight consecutive elements at column c of a row as they lie in memory: one
// 16-byte piece of bf16 or two of fp32.
template <bool NT>
__device__ __forceinline__ void raw8(const void* base, bool bf16, int64_t off, uint32_t c, u32x4 (&q)[2]) {
  const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(base) + (off + c) * (bf16 ? 2 : 4));
  q[0] = NT ? __builtin_nontemporal_load(p) : p[0];
  if (!bf16) q[1] = NT ? __builtin_nontemporal_load(p + 1) : p[1];
}

__device__ __forceinline__ u32x4 vec8(const void* base, int64_t off, uint32_t c) {
  return *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + off + c);
}

__device__ __forceinline__ void widen(u32x4 q, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = bf16_lo(q[j]);
    v[2 * j + 1] = bf16_hi(q[j]);
  }
}

__device__ __forceinline__ void widen8(const u32x4 (&q)[2], bool bf16, float (&v)[8]) {
  if (bf16) {
    widen(q[0], v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(q[j >> 2][j & 3]);
  }
}

// The same, widened (columns past d read as 0;
// VEC: whole aligned chunks).
template <bool VEC, bool NT = false>
__device__ __forceinline__ void load8(const void* base, bool bf16, int64_t off, uint32_t c, uint32_t d, float (&v)[8]) {
  if constexpr (VEC) {
    if (bf16) {
      const u32x4* qp = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + off + c);
      widen(NT ? __builtin_nontemporal_load(qp) : *qp, v);
    } else {
      const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(base) + off + c);
      const f32x4 a = NT ? __builtin_nontemporal_load(p) : p[0], b = NT ? __builtin_nontemporal_load(p + 1) : p[1];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = 0.0f;
      if (c + j < d)
        v[j] = bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(base)[off + c + j] << 16)
                    : static_cast<const float*>(base)[off + c + j];
    }
  }
}

template <bool VEC, bool NT>
__device__ __forceinline__ void store8(void* base, bool bf16, int64_t off, uint32_t c, uint32_t d, const float (&v)[8]) {
  if constexpr (VEC) {
    if (bf16) {
      u32x4* qp = reinterpret_cast<u32x4*>(static_cast<uint16_t*>(base) + off + c);
      const u32x4 q = u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
      if constexpr (NT) __builtin_nontemporal_store(q, qp);
      else *qp = q;
    } else {
      f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(base) + off + c);
      const f32x4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
      if constexpr (NT) __builtin_nontemporal_store(a, p), __builtin_nontemporal_store(b, p + 1);
      else p[0] = a, p[1] = b;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (c + j >= d) continue;
      if (bf16) static_cast<uint16_t*>(base)[off + c + j] = (uint16_t)pack_bf16(v[j], 0.0f);
      else static_cast<float*>(base)[off + c + j] = v[j];
    }
  }
}

// Lane i's value from lane i ^ 1 or i ^ 2 of its quad.
template <int X>
__device__ __forceinline__ float quad_xor(float v) {
  constexpr int ctrl = X == 1 ? 0xB1 : 0x4E;   // quad_perm [1,0,3,2] / [2,3,0,1]
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), ctrl, 0xF, 0xF, true));
}

__device__ __forceinline__ float row_sum(float v, float* slot, int wave, int waves) {
  v += quad_xor<1>(v);
  v += quad_xor<2>(v);
  v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x141, 0xF, 0xF, true));   // row_half_mirror
  v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x140, 0xF, 0xF, true));   // row_mirror
  // both results hold v's even and odd 16-lane rows, then its lower and upper halves
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(h[0]) + __uint_as_float(h[1]);
  if (waves > 1) {
    if ((threadIdx.x & 63) == 0) slot[wave] = v;
    __syncthreads();
    v = slot[0];
    for (int i = 1; i < waves; ++i) v += slot[i];
  }
  return v;
}

// v minus the row's mean (columns past d stay 0).
template <int EPL, bool VEC>
__device__ __forceinline__ void centre(const NormArgs& a, float (&v)[EPL][8], uint32_t c0, uint32_t step, float inv_d,
                                       float* slots, int wave, int waves) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < EPL; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) s += v[i][j];
  const float mean = row_sum(s, slots, wave, waves) * inv_d;
#pragma unroll
  for (int i = 0; i < EPL; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = c0 + i * step + (VEC ? 0 : j) < a.d ? v[i][j] - mean : 0.0f;
}

// mean(v^2) + eps
template <int EPL>
__device__ __forceinline__ float mean_square(const float (&v)[EPL][8], float inv_d, float eps, float* slots, int wave,
                                             int waves) {
  float q = 0.0f;
#pragma unroll
  for (int i = 0; i < EPL; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) q = __builtin_fmaf(v[i][j], v[i][j], q);
  return __builtin_fmaf(row_sum(q, slots, wave, waves), inv_d, eps);
}

// The scale of norm(v) over the row's d elements; centres v for a layer norm.
//
// The mean square of fp32 values leaves fp32's range long before they do, and
// v_rsq_f32 takes subnormal arguments as 0.  Where it falls below 2^-100 (only
// with eps below that; down to there underflow costs its squares nothing) or
// overflows, the row is scaled by 2^100 or 2^-100, centred again (the first mean
// was rounded to a multiple of 2^-149) and squared anew: 2^-149 <= |v| < 2^-42
// gives squares in [2^-98, 2^116], |v| < 2^128 squares below 2^56.  What is
// returned is then the scale of the scaled row.  Every lane holds the same sum,
// so a workgroup's waves take the same way.  (A block of its own: as a second
// pass of a loop it took 13 more registers and spilled long rows.)
template <int EPL, bool VEC>
__device__ __forceinline__ float statistics(const NormArgs& a, float (&v)[EPL][8], uint32_t c0, uint32_t step,
                                            float* slots, int wave, int waves) {
  const float inv_d = 1.0f / (float)a.d;
  if (a.layer) centre<EPL, VEC>(a, v, c0, step, inv_d, slots, wave, waves);
  float ms = mean_square(v, inv_d, a.eps, slots + MAXW, wave, waves);
  const float t = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(ms)));
  if (__builtin_expect(t < 0x1p-100f || t == __builtin_inff(), 0)) {
    const float s = t < 1.0f ? 0x1p100f : 0x1p-100f;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= s;
    if (waves > 1) __syncthreads();   // the slots have been read
    if (a.layer) centre<EPL, VEC>(a, v, c0, step, inv_d, slots, wave, waves);
    ms = mean_square(v, inv_d, a.eps * s * s, slots + MAXW, wave, waves);
  }
  return __builtin_amdgcn_rsqf(ms);
}

__device__ __forceinline__ int tiled_swz(int r) { return ((r >> 1) ^ (r >> 2)) & 3; }

// Where block `blk` of a row goes.
struct BlockOut {
  uint8_t* code;    // 16 bytes
  uint8_t* scale;
};

__device__ __forceinline__ BlockOut block_out(const NormArgs& a, uint32_t row, uint32_t blk) {
  if (a.tiled) {
    const uint32_t r = row % kTileRows, cb = blk & 3u;
    const uint64_t ts = (uint64_t)(row / kTileRows) * (a.d >> 7) + (blk >> 2);
    return {a.codes + ts * (kTileRows * 64) + r * 64 + 16 * (cb ^ tiled_swz((int)r)),
            a.scales + ts * (kTileRows * 4) + r * 4 + cb};
  }
  const uint64_t b = (uint64_t)row * (a.d >> 5) + blk;
  return {a.codes + 16 * b, a.scales + b};
}

// Quantizes one chunk per lane; the four lanes of a quad hold one block.
template <int ROT>
__device__ __forceinline__ void quantize_quad(const NormArgs& a, float (&v)[8], uint32_t row, uint32_t c, int lane) {
  if constexpr (ROT == 3) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] * a.fa[c + j];
  }
  if constexpr (ROT == 1) {
#pragma unroll
    for (int h = 1; h < 8; h <<= 1)
#pragma unroll
      for (int i = 0; i < 8; i += 2 * h)
#pragma unroll
        for (int j = i; j < i + h; ++j) {
          const float u = v[j], w = v[j + h];
          v[j] = u + w;
          v[j + h] = u - w;
        }
    // strides 8 and 16 across the quad: the lower lane forms u + w, the upper
    // one u - w from its partner's u
    const uint32_t s1 = (lane & 1) ? 0x80000000u : 0u, s2 = (lane & 2) ? 0x80000000u : 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = quad_xor<1>(v[j]) + __uint_as_float(__float_as_uint(v[j]) ^ s1);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = quad_xor<2>(v[j]) + __uint_as_float(__float_as_uint(v[j]) ^ s2);
    const float k = __uint_as_float(0x3E3504F3u);   // nearest fp32 to 1/sqrt(32)
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] * k;
  }
  float am = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) am = fmaxf(am, fabsf(v[j]));
  am = fmaxf(am, quad_xor<1>(am));
  am = fmaxf(am, quad_xor<2>(am));
  const uint32_t sbyte = sbyte_of_amax(am);
  const float scale = scale_of(sbyte);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
  if (c >= a.d) return;
  const BlockOut o = block_out(a, row, c >> 5);
  reinterpret_cast<uint32_t*>(o.code)[lane & 3] = w;
  if ((lane & 3) == 0) *o.scale = (uint8_t)sbyte;
}

// One Kronecker-transformed block over Q lanes: lane k forms column k of both
// stages, U[j][k] for every j and then y[Q i + k] -- the chains of the one-lane
// transform in their order -- and the group merges the block amax and the code
// nibbles with butterflies (an exact max and an OR).
template <int P, int Q>
__device__ __forceinline__ void kron_block(const NormArgs& a, const float* blk, uint32_t row, uint32_t b, int k) {
  float u[P];
#pragma unroll
  for (int j = 0; j < P; ++j) u[j] = a.fb[k * Q] * blk[Q * j];
#pragma unroll
  for (int l = 1; l < Q; ++l) {
    const float f = a.fb[k * Q + l];
#pragma unroll
    for (int j = 0; j < P; ++j) u[j] = __builtin_fmaf(f, blk[Q * j + l], u[j]);
  }
  auto out = [&](int i) {   // y[Q i + k]
    float acc = a.fa[i * P] * u[0];
#pragma unroll
    for (int j = 1; j < P; ++j) acc = __builtin_fmaf(a.fa[i * P + j], u[j], acc);
    return acc;
  };
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  float am = 0.0f, scale;
  uint32_t sbyte;
  auto put = [&](int i, float v) {   // its code, into nibble Q i + k of the block
    const int e = Q * i + k;
    const uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v, 0.0f, scale, 0) & 0xFu;
    const uint32_t sh = 4u * (uint32_t)(e & 7);
#pragma unroll
    for (int d = 0; d < 4; ++d) w[d] |= (e >> 3) == d ? c << sh : 0u;
  };
  if constexpr (P == 32) {
    // a 32 x 32 first factor: rolled loops that form each value twice, since
    // its 1024 values, loaded ahead by an unrolled loop, spill
#pragma unroll 1
    for (int i = 0; i < P; ++i) am = fmaxf(am, fabsf(out(i)));
    sbyte = sbyte_of_amax(am);
    scale = scale_of(sbyte);
#pragma unroll 1
    for (int i = 0; i < P; ++i) put(i, out(i));
  } else {
    float y[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      y[i] = out(i);
      am = fmaxf(am, fabsf(y[i]));
    }
#pragma unroll
    for (int o = 1; o < Q; o <<= 1) am = fmaxf(am, __shfl_xor(am, o));
    sbyte = sbyte_of_amax(am);
    scale = scale_of(sbyte);
#pragma unroll
    for (int i = 0; i < P; ++i) put(i, y[i]);
  }
#pragma unroll
  for (int o = 1; o < Q; o <<= 1) {
#pragma unroll
    for (int d = 0; d < 4; ++d) w[d] |= (uint32_t)__shfl_xor((int)w[d], o);
  }
  if (k != 0) return;
  const BlockOut o = block_out(a, row, b);
  *reinterpret_cast<uint4*>(o.code) = make_uint4(w[0], w[1], w[2], w[3]);
  *o.scale = (uint8_t)sbyte;
}

// OUT: 0 dense y (or none), 1 MXFP4.  ROT as in block_quant.h; P x Q the
// Kronecker factors, KD their columns in LDS.  EPL chunks of 8 columns per lane,
// 512 EPL columns per wave.  NT: non-temporal loads and stores of whole rows.
template <int EPL, bool VEC, bool NT, int OUT, int ROT, int P, int Q, int KD>
__global__ __launch_bounds__(64 * MAXW) void norm_kernel(NormArgs a) {
  // Kronecker: the row, 36 words per 32-element block
  __shared__ __attribute__((aligned(16))) float krow[KD / 32 * 36 + 1];
  __shared__ float slots[4 * MAXW];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  // Tiled codes of 16 rows share cache lines, and workgroup i runs on XCD i % 8,
  // each with its own L2: an XCD takes 32 neighbouring rows of 256 (57344 x 3072
  // with modulation, H32: 162 us against 167).
  uint32_t row = a.row0 + blockIdx.x;
  if (OUT == 1 && a.tiled && (row | 255u) < a.rows) row = (row & ~255u) + 32 * (row & 7) + ((row >> 3) & 31);
  const uint32_t c0 = 8 * threadIdx.x, step = 512 * waves;
  const int64_t voff = (a.gate != nullptr || a.scale != nullptr || a.shift != nullptr)
                           ? (int64_t)(row / a.group_rows) * a.ld_vec
                           : 0;

  // All of x's chunks are in flight before the first is widened.
  constexpr bool AHEAD = VEC && EPL <= 2;
  const bool ahead = AHEAD && a.vec_bf16;
  constexpr int PE = AHEAD ? EPL : 1;
  u32x4 xq[PE][2], last[4][PE];
  if constexpr (AHEAD) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const uint32_t c = c0 + i * step;
      if (c < a.d) raw8<NT>(a.x, a.x_bf16, (int64_t)row * a.ld_x, c, xq[i]);
    }
  }
  auto vec = [&](int which, const void* base, int64_t off, int i, uint32_t c, float (&w)[8]) {
    if (AHEAD && ahead) widen(last[which][AHEAD ? i : 0], w);
    else load8<VEC>(base, a.vec_bf16, off, c, a.d, w);
  };

  float v[EPL][8];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const uint32_t c = c0 + i * step;
    if (c >= a.d) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    } else if constexpr (AHEAD) {
      widen8(xq[i], a.x_bf16, v[i]);
    } else {
      load8<VEC, NT>(a.x, a.x_bf16, (int64_t)row * a.ld_x, c, a.d, v[i]);
    }
  }
  if (a.post_norm) {
    const float inv = statistics<EPL, VEC>(a, v, c0, step, slots, wave, waves);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const uint32_t c = c0 + i * step;
      if (c >= a.d) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= inv;
      if (a.post_weight != nullptr) {
        float w[8];
        load8<VEC>(a.post_weight, a.vec_bf16, 0, c, a.d, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= w[j];
      }
    }
  }
  if (a.gate != nullptr || a.residual != nullptr || a.residual_out != nullptr) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const uint32_t c = c0 + i * step;
      if (c >= a.d) continue;
      if (a.gate != nullptr) {
        float w[8];
        load8<VEC>(a.gate, a.vec_bf16, voff, c, a.d, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= w[j];
      }
      if (a.residual != nullptr) {
        float w[8];
        load8<VEC, NT>(a.residual, a.r_bf16, (int64_t)row * a.ld_r, c, a.d, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = __builtin_fmaf(a.residual_scale, w[j], v[i][j]);
      }
      if (a.residual_out != nullptr) store8<VEC, NT>(a.residual_out, a.r_bf16, (int64_t)row * a.ld_ro, c, a.d, v[i]);
    }
  }
  if (OUT == 0 && a.y == nullptr) return;

  // The last step's vectors are asked for before the statistics' barriers: an
  // L2 round trip for all of them, hidden, instead of one each behind the
  // barriers (57344 x 3072 with modulation to bf16: 132 us against 161, together
  // with x's chunks above).  Asked for with x they would take the registers of
  // a resident workgroup (173 us).
  if constexpr (AHEAD) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const uint32_t c = c0 + i * step;
      if (!ahead || c >= a.d) continue;
      if (a.weight != nullptr) last[0][i] = vec8(a.weight, 0, c);
      if (a.bias != nullptr) last[1][i] = vec8(a.bias, 0, c);
      if (a.scale != nullptr) last[2][i] = vec8(a.scale, voff, c);
      if (a.shift != nullptr) last[3][i] = vec8(a.shift, voff, c);
    }
  }
  const float inv = statistics<EPL, VEC>(a, v, c0, step, slots + 2 * MAXW, wave, waves);
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const uint32_t c = c0 + i * step;
    // a lane past the row's end has no quad partner inside it (d % 32 == 0)
    if (c < a.d) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= inv;
      if (a.weight != nullptr) {
        float w[8];
        vec(0, a.weight, 0, i, c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= w[j];
      }
      if (a.bias != nullptr) {
        float w[8];
        vec(1, a.bias, 0, i, c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += w[j];
      }
      if (a.scale != nullptr) {
        float w[8];
        vec(2, a.scale, voff, i, c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= 1.0f + w[j];
      }
      if (a.shift != nullptr) {
        float w[8];
        vec(3, a.shift, voff, i, c, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += w[j];
      }
    }
    if constexpr (OUT == 0) {
      if (c < a.d) store8<VEC, NT>(a.y, a.y_bf16, (int64_t)row * a.ld_y, c, a.d, v[i]);
    } else if constexpr (ROT != 2) {
      if (c < a.d) quantize_quad<ROT>(a, v[i], row, c, lane);
    } else {
      if (c < a.d) {
        float4* p = reinterpret_cast<float4*>(krow + (c >> 5) * 36 + (c & 31));
        p[0] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
        p[1] = make_float4(v[i][4], v[i][5], v[i][6], v[i][7]);
      }
    }
  }
  if constexpr (OUT == 1 && ROT == 2) {
    __syncthreads();
    const uint32_t nblk = a.d >> 5;
    const uint32_t per = blockDim.x / Q;   // blocks a pass
    for (uint32_t b0 = 0; b0 < nblk; b0 += per) {
      const uint32_t b = b0 + threadIdx.x / Q;
      if (b < nblk) kron_block<P, Q>(a, krow + b * 36, row, b, lane % Q);   // whole groups of Q lanes
    }
  }
}

template <int EPL, bool VEC, bool NT, int OUT, int ROT, int P = 1, int Q = 32, int KD = 0>
void run(const NormArgs& a, hipStream_t s) {
  const uint32_t waves = (a.d + 512 * EPL - 1) / (512 * EPL);
  // A grid holds fewer than 2^32 threads: more rows take several launches, of
  // whole groups of 256 rows.
  const uint32_t per = 0xFFFFFFFFu / (64 * waves) & ~255u;
  for (uint32_t row0 = 0; row0 < a.rows; row0 += per) {
    NormArgs b = a;
    b.row0 = row0;
    norm_kernel<EPL, VEC, NT, OUT, ROT, P, Q, KD><<<std::min(per, a.rows - row0), 64 * waves, 0, s>>>(b);
  }
}

// Chunks per lane.  Few rows (two workgroups per CU): one, the most waves and
// the shortest row latency (16 x 4096: 3.4 us against 4.0 with two; 3.1 since
// the last step's vectors are read ahead).  More: two, which ask for twice the
// bytes per wave before the first barrier (57344 x 3072 with modulation 255 us
// against 318; 243 since then).  Rows past two chunks on 16 waves: eight.
// Either way a row takes as many waves as it has whole 512-column chunks for:
// with four waves always, 3072 columns left half of the second chunk idle (301).
template <bool VEC, bool NT, int OUT, int ROT>
void run_width(const NormArgs& a, hipStream_t s) {
  if (a.d <= 8192 && a.rows <= 2u * (uint32_t)cu_count()) run<1, VEC, NT, OUT, ROT>(a, s);
  else if (a.d <= 16384) run<2, VEC, NT, OUT, ROT>(a, s);
  else run<8, VEC, NT, OUT, ROT>(a, s);
}

// Inputs larger than the 256 MB last-level cache stream past it (263 -> 253 us
// at 57344 x 3072); smaller ones, which the kernel before has just written,
// are read through it (777 x 5120: 12.6 us against 15.5).
template <bool VEC, int OUT, int ROT>
void run_size(const NormArgs& a, hipStream_t s) {
  const uint64_t elem = (a.x_bf16 ? 2 : 4) + (a.residual == nullptr ? 0 : a.r_bf16 ? 2 : 4);
  if (a.rows * elem * a.d > (uint64_t(256) << 20)) run_width<VEC, true, OUT, ROT>(a, s);
  else run_width<VEC, false, OUT, ROT>(a, s);
}

template <int P, int Q>
void run_kron(const NormArgs& a, hipStream_t s) {
  if (a.d <= 4096) run<2, true, false, 1, 2, P, Q, 4096>(a, s);
  else run<2, true, false, 1, 2, P, Q, kNormMaxDKron>(a, s);
}

hipError_t dispatch(const NormArgs& a, hipStream_t s) {
  if (a.codes == nullptr) {
    if (a.vec) run_size<true, 0, 0>(a, s);
    else run_width<false, false, 0, 0>(a, s);
    return hipGetLastError();
  }
  switch (a.rot) {
    case 0: run_size<true, 1, 0>(a, s); break;
    case 1: run_size<true, 1, 1>(a, s); break;
    case 3: run_size<true, 1, 3>(a, s); break;
    default:
      switch (a.p) {
        case 1: run_kron<1, 32>(a, s); break;
        case 2: run_kron<2, 16>(a, s); break;
        case 4: run_kron<4, 8>(a, s); break;
        case 8: run_kron<8, 4>(a, s); break;
        case 16: run_kron<16, 2>(a, s); break;
        case 32: run_kron<32, 1>(a, s); break;
        default: return hipErrorInvalidValue;
      }
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  return dispatch(a, s);
}

}  // namespace mxfp4
