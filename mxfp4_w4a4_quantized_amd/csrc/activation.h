// Activations of the feed-forward epilogues, fp32 in and out.
//
// Transcendentals run at a quarter of the VALU rate, so each activation is
// written with one exponential and one reciprocal (v_exp_f32 and v_rcp_f32,
// 1 ulp each), and constants are folded into the exponent's base 2.
//   silu(x)      = x / (1 + 2^(-log2(e) x))
//   gelu_tanh(x) = 0.5 x (1 + tanh(u)) = x sigmoid(2 u),
//                  2 u = 2 sqrt(2/pi) (x + 0.044715 x^3)
//   gelu(x)      = x Phi(x), Phi(-a) = t poly(t) e^(-a^2 / 2) for a >= 0 with
//                  t = 1 / (1 + 0.295 a): a polynomial of degree 7 fitted to
//                  Phi(-a) e^(a^2 / 2) / t for a <= 13.5 (in 64 bits, by least
//                  squares reweighted towards the largest error, in units of
//                  (3 + 1.25 a^2) 2^-24 of the value, what rounding the exponent
//                  costs).  The tail keeps its relative accuracy, (45 + 1.5 x^2)
//                  2^-24 at most; the last factor is the exponential, which stays
//                  normal as long as the result does.
// At infinities and NaN they follow the formulas: the exponential saturates to
// 0 or infinity, and act(-inf) is -inf * 0 = NaN.
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>

namespace mxfp4 {
namespace act {

constexpr int NONE = 0, RELU = 1, SILU = 2, GELU = 3, GELU_TANH = 4;   // mxfp4_act

__device__ __forceinline__ float relu(float x) { return x < 0.0f ? 0.0f : x; }   // keeps NaN

// x / (1 + 2^t) with both sides of the quotient scaled by 2^-24 (one multiply
// more): v_rcp_f32 flushes results below 2^-126, which 1 / (1 + 2^t) reaches
// while x times it is still a normal number.
__device__ __forceinline__ float over_one_plus_exp2(float x, float t) {
  constexpr float c = 1.0f / 16777216.0f;
  return (x * c) * __builtin_amdgcn_rcpf(__builtin_fmaf(__builtin_amdgcn_exp2f(t), c, c));
}

__device__ __forceinline__ float silu(float x) { return over_one_plus_exp2(x, x * -1.442695040889f); }

__device__ __forceinline__ float gelu_tanh(float x) {
  // -log2(e) * 2 sqrt(2/pi) and that times 0.044715
  return over_one_plus_exp2(x, x * __builtin_fmaf(-0.10294324f, x * x, -2.3022082f));
}

__device__ __forceinline__ float gelu(float x) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(fabsf(x), 0.295f, 1.0f));
  float p = __builtin_fmaf(t, 0.0373435728f, -0.173062041f);
  p = __builtin_fmaf(t, p, 0.249138921f);
  p = __builtin_fmaf(t, p, -0.0914765298f);
  p = __builtin_fmaf(t, p, 0.148233667f);
  p = __builtin_fmaf(t, p, 0.0925811902f);
  p = __builtin_fmaf(t, p, 0.119663447f);
  p = __builtin_fmaf(t, p, 0.117577776f);
  const float e = __builtin_amdgcn_exp2f(x * x * -0.7213475204f);   // e^(-x^2 / 2); NaN stays NaN
  // s e = x Phi(-|x|), in s with x at most 2^100 (so that it is 0 at infinity);
  // then x Phi(x) = max(x, 0) - |s e|.  Both limits on x's bits: as floats each
  // would cost the compiler an instruction more for signalling NaN.
  const int i = __float_as_int(x);
  const float s = __int_as_float(min(i, 0x71800000)) * (p * t);
  return __builtin_fmaf(-fabsf(s), e, __int_as_float(max(i, 0)));
}

}  // namespace act
}  // namespace mxfp4
