// Argument checks shared by the C-ABI files (api.cpp, api_ffn.cpp, api_moe.cpp).
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

inline bool is_dtype(int32_t t) { return t == MXFP4_F32 || t == MXFP4_BF16; }
inline int64_t size_of(int32_t t) { return t == MXFP4_BF16 ? 2 : 4; }
inline bool is_layout(int32_t l) { return l == MXFP4_LAYOUT_ROWMAJOR || l == MXFP4_LAYOUT_TILED; }
inline bool is_act(int32_t a) { return a >= MXFP4_ACT_NONE && a <= MXFP4_ACT_GELU_TANH; }

inline bool sizes_ok(int64_t m, int64_t n, int64_t k, int32_t layout) {
  return m >= 0 && n >= 0 && k > 0 && (k % (layout == MXFP4_LAYOUT_TILED ? kTileK : 32)) == 0;
}

// Where a GEMM with an epilogue writes its result, dense or packed.
inline mxfp4_status dense_output(void* y, int32_t y_dtype, int64_t ld_y, FusedArgs& f) {
  if (y == nullptr) return MXFP4_ERR_INVALID_ARG;
  if (!aligned(y, size_of(y_dtype))) return MXFP4_ERR_UNSUPPORTED;
  f.g.y = y;
  f.g.ld_y = ld_y;
  f.g.y_bf16 = y_dtype == MXFP4_BF16;
  return MXFP4_OK;
}

inline mxfp4_status packed_output(const Rot& r, uint8_t* y_codes, uint8_t* y_scales, int32_t y_layout, int64_t n,
                           FusedArgs& f) {
  if (y_codes == nullptr || y_scales == nullptr) return MXFP4_ERR_INVALID_ARG;
  if (r.kind != MXFP4_ROT_NONE && r.kind != MXFP4_ROT_HADAMARD32) return MXFP4_ERR_UNSUPPORTED;
  const bool q_tiled = y_layout == MXFP4_LAYOUT_TILED;
  if ((n % (q_tiled ? kTileK : 32)) != 0) return MXFP4_ERR_UNSUPPORTED;
  if (!aligned(y_codes, 16) || !aligned(y_scales, 4)) return MXFP4_ERR_UNSUPPORTED;
  f.g.y = nullptr;
  f.g.ld_y = n;
  f.g.y_bf16 = false;
  f.g.q_out = true;
  f.g.q_tiled = q_tiled;
  f.g.q_codes = y_codes;
  f.g.q_scales = y_scales;
  f.h32 = r.kind == MXFP4_ROT_HADAMARD32;
  return MXFP4_OK;
}

}  // namespace args
}  // namespace mxfp4
