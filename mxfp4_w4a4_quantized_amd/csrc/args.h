// Argument checks shared by the C-ABI files (api.cpp, api_ffn.cpp).
#pragma once
#include "mxfp4.h"

#include <cstdint>

#include "internal.h"

namespace mxfp4 {
namespace args {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline mxfp4_status from_hip(hipError_t e) { return e == hipSuccess ? MXFP4_OK : MXFP4_ERR_HIP; }

constexpr int64_t kMaxDim = int64_t(1) << 30;

struct Rot {
  int32_t kind = MXFP4_ROT_NONE, p = 0, q = 0;
  const float* fa = nullptr;
  const float* fb = nullptr;
};

// Validates a rotation descriptor (NULL = none).
inline mxfp4_status parse_rotation(const mxfp4_rotation* rot, Rot& r) {
  if (rot == nullptr) return MXFP4_OK;
  r.kind = rot->kind;
  if (r.kind != MXFP4_ROT_NONE && r.kind != MXFP4_ROT_HADAMARD32 && r.kind != MXFP4_ROT_KRON &&
      r.kind != MXFP4_ROT_SMOOTH)
    return MXFP4_ERR_INVALID_ARG;
  if (rot->reserved != 0) return MXFP4_ERR_INVALID_ARG;
  if (r.kind == MXFP4_ROT_KRON) {
    r.p = rot->p;
    r.q = rot->q;
    if (r.p < 1 || r.q < 1 || r.p * r.q != 32 || (r.p & (r.p - 1)) != 0) return MXFP4_ERR_INVALID_ARG;
    if (rot->a == nullptr || rot->b == nullptr) return MXFP4_ERR_INVALID_ARG;
    r.fa = rot->a;
    r.fb = rot->b;
    if (!aligned(r.fa, 4) || !aligned(r.fb, 4)) return MXFP4_ERR_UNSUPPORTED;
  }
  if (r.kind == MXFP4_ROT_SMOOTH) {
    if (rot->a == nullptr) return MXFP4_ERR_INVALID_ARG;
    r.fa = rot->a;
    if (!aligned(r.fa, 16)) return MXFP4_ERR_UNSUPPORTED;
  }
  return MXFP4_OK;
}

}  // namespace args
}  // namespace mxfp4
