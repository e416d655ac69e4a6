// What the experts' products read of a plan on the device.
#pragma once
#include "internal.h"
#include "moe_plan.h"

namespace mxfp4 {
namespace moe {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// Scalar loads of what an earlier kernel wrote, at wave-uniform addresses: they
// are not counted among the vector loads that the GEMMs keep in flight.
__device__ __forceinline__ int uniform(const int32_t* p) {
  return *(const __attribute__((address_space(4))) int32_t*)(uintptr_t)p;
}
__device__ __forceinline__ i32x4 uniform4(const int32_t* p) {
  return *(const __attribute__((address_space(4))) i32x4*)(uintptr_t)p;
}

// The arguments of a row tile's product: its expert's weights and biases, its
// last row as the end of the rows.  Returns its first row.
__device__ __forceinline__ int enter_tile(const MoeArgs& a, FusedArgs& f, const i32x4& t, int tile, int rows) {
  const int64_t e = t[0];
  f.g.b_codes = a.g.b_codes + e * a.w_codes;
  f.g.b_scales = a.g.b_scales + e * a.w_scales;
  const int64_t bias = e * a.g.n * (a.vec_bf16 ? 2 : 4);
  if (a.bias != nullptr) f.bias = static_cast<const uint8_t*>(a.bias) + bias;
  if (a.glu) {
    f.u_codes = a.u_codes + e * a.w_codes;
    f.u_scales = a.u_scales + e * a.w_scales;
    if (a.bias_u != nullptr) f.bias_u = static_cast<const uint8_t*>(a.bias_u) + bias;
  }
  f.g.m = t[2];
  return t[1] + (tile - t[3]) * rows;
}

// Row of A that row p of the result reads: with experts, the plan's token.
__device__ __forceinline__ int source_row(const FusedArgs&, int p) { return p; }
// The layout of A, and the bytes from one expert's weights to the next's.
__device__ __forceinline__ bool a_tiled(const FusedArgs& a) { return a.g.tiled; }
__device__ __forceinline__ bool a_tiled(const MoeArgs& a) { return a.a_tiled; }
__device__ __forceinline__ int64_t code_step(const FusedArgs&) { return 0; }
__device__ __forceinline__ int64_t code_step(const MoeArgs& a) { return a.w_codes; }
__device__ __forceinline__ int64_t scale_step(const FusedArgs&) { return 0; }
__device__ __forceinline__ int64_t scale_step(const MoeArgs& a) { return a.w_scales; }
__device__ __forceinline__ int source_row(const MoeArgs& a, int p) { return a.token != nullptr ? a.token[p] : p; }

}  // namespace moe
}  // namespace mxfp4
