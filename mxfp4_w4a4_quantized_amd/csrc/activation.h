// Activations of the feed-forward epilogues, fp32 in and out.
//
// Transcendentals run at a quarter of the VALU rate, so each activation is
// written with one exponential and one reciprocal (v_exp_f32 and v_rcp_f32,
// 1 ulp each), and constants are folded into the exponent's base 2.
//   silu(x)      = x / (1 + 2^(-log2(e) x))
//   gelu_tanh(x) = 0.5 x (1 + tanh(u)) = x sigmoid(2 u),
//                  2 u = 2 sqrt(2/pi) (x + 0.044715 x^3)
//   gelu(x)      = x Phi(x), Phi by Abramowitz and Stegun 7.1.26: for z >= 0
//                  erfc(z) = t (a1 + t (a2 + t (a3 + t (a4 + t a5)))) e^(-z^2),
//                  t = 1 / (1 + 0.3275911 z), absolute error below 1.5e-7
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
  const float ax = fabsf(x);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(ax, 0.231641888f, 1.0f));   // 0.3275911 / sqrt(2)
  // the coefficients halved: p e = erfc(|x| / sqrt(2)) / 2 = Phi(-|x|)
  float p = __builtin_fmaf(t, 0.5307027145f, -0.7265760135f);
  p = __builtin_fmaf(t, p, 0.7107068705f);
  p = __builtin_fmaf(t, p, -0.142248368f);
  p = __builtin_fmaf(t, p, 0.127414796f);
  const float q = p * t * __builtin_amdgcn_exp2f(x * x * -0.7213475204f);   // e^(-x^2 / 2)
  return x * (x < 0.0f ? q : 1.0f - q);
}

}  // namespace act
}  // namespace mxfp4
