// Activations of the feed-forward epilogues, fp32 in and out.
//
// Transcendentals run at a quarter of the VALU rate, so each activation is
// written with one exponential and one reciprocal (v_exp_f32 and v_rcp_f32,
// 1 ulp each), and constants are folded into the exponent's base 2.  Relative to
// the result, wherever that is a normal number, silu and the tanh GELU are off
// by at most (4 |t| + 10) 2^-24, t the exponent: its rounding grows with it.
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
// 0 or infinity, and act(-inf) is -inf * 0 = NaN.  Each takes a lane's values
// together.
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>

namespace mxfp4 {
namespace act {

constexpr int NONE = 0, RELU = 1, SILU = 2, GELU = 3, GELU_TANH = 4;   // mxfp4_act

// silu and the tanh GELU are x / (1 + 2^t) with t by the functions below; t stays
// below 126 down to the x that has the bits `deep`.
struct Silu {
  static constexpr uint32_t deep = 0xC2AE0000u;   // -87
  static __device__ __forceinline__ float t(float x) { return x * -1.442695040889f; }
};
struct GeluTanh {
  static constexpr uint32_t deep = 0xC11E6666u;   // -9.9
  // -log2(e) * 2 sqrt(2/pi) and that times 0.044715
  static __device__ __forceinline__ float t(float x) { return x * __builtin_fmaf(-0.10294324f, x * x, -2.3022082f); }
};

// x * rcp(1 + 2^t) is right where that reciprocal is a normal number: v_rcp_f32
// flushes below 2^-126, and past t = 128 the exponential is infinite, while the
// result stays normal to t = 133 (silu at -92).  No real pre-activation gets
// there, so the other form stands behind a branch that a wave takes only if one
// of its values needs it, found with an integer maximum of three values an
// instruction; scaling both sides of every quotient instead costs each value a
// multiply, and loses the smallest values' bits.
template <class A, int N>
__device__ __forceinline__ void over_one_plus_exp2(float (&v)[N]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) top = max(top, __float_as_uint(v[i]));
  // (negative floats order like their bits; negative NaN takes the branch too)
  if (__builtin_expect(__builtin_amdgcn_ballot_w64(top > A::deep) == 0, 1)) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = v[i] * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(A::t(v[i])));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      // past t = 64 the quotient is x 2^-t
      const float t = A::t(v[i]);
      const bool far = t > 64.0f;
      const float e = __builtin_amdgcn_exp2f(far ? 64.0f - t : t);
      const float r = __builtin_amdgcn_rcpf(1.0f + e);
      v[i] = (v[i] * (far ? e : 1.0f)) * (far ? 0x1p-64f : r);
      __builtin_amdgcn_sched_barrier(0);   // one value at a time: few registers
    }
  }
}

__device__ __forceinline__ float gelu_one(float x) {
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

template <int N>
__device__ __forceinline__ void relu(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i];   // keeps NaN
}
template <int N>
__device__ __forceinline__ void silu(float (&v)[N]) { over_one_plus_exp2<Silu>(v); }
template <int N>
__device__ __forceinline__ void gelu_tanh(float (&v)[N]) { over_one_plus_exp2<GeluTanh>(v); }
template <int N>
__device__ __forceinline__ void gelu(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = gelu_one(v[i]);
}

}  // namespace act
}  // namespace mxfp4
