// C-ABI of the feed-forward operators: argument validation, kernel selection,
// HIP error mapping.  The declarations and error behaviour are documented in
// mxfp4.h.
#include "mxfp4.h"

#include <cmath>
#include <cstdint>

#include "args.h"

using namespace mxfp4::args;

namespace {

// Validates a norm descriptor and fills the kernel's arguments.  rows == 0
// passes with only the sizes and enums checked.
mxfp4_status parse_norm(const mxfp4_norm_args* a, bool dense, mxfp4::NormArgs& k) {
  if (a == nullptr || a->reserved != 0) return MXFP4_ERR_INVALID_ARG;
  if (a->kind != MXFP4_NORM_RMS && a->kind != MXFP4_NORM_LAYER) return MXFP4_ERR_INVALID_ARG;
  if (!is_dtype(a->x_dtype) || !is_dtype(a->r_dtype) || !is_dtype(a->vec_dtype)) return MXFP4_ERR_INVALID_ARG;
  if (a->rows < 0 || a->d < 1 || a->ld_x < a->d) return MXFP4_ERR_INVALID_ARG;
  if (a->residual != nullptr && a->ld_r < a->d) return MXFP4_ERR_INVALID_ARG;
  if (a->residual_out != nullptr && a->ld_ro < a->d) return MXFP4_ERR_INVALID_ARG;
  if (a->post_weight != nullptr && a->post_norm == 0) return MXFP4_ERR_INVALID_ARG;
  const bool grouped = a->gate != nullptr || a->scale != nullptr || a->shift != nullptr;
  if (grouped && (a->group_rows < 1 || a->ld_vec < a->d)) return MXFP4_ERR_INVALID_ARG;
  if (!(a->eps >= 0.0f) || !std::isfinite(a->eps)) return MXFP4_ERR_INVALID_ARG;
  if (a->rows == 0) return MXFP4_OK;
  if (a->x == nullptr) return MXFP4_ERR_INVALID_ARG;
  if (a->d > mxfp4::kNormMaxD || a->rows >= kMaxDim) return MXFP4_ERR_UNSUPPORTED;
  const int64_t xs = size_of(a->x_dtype), rs = size_of(a->r_dtype), vs = size_of(a->vec_dtype);
  const void* vecs[6] = {a->post_weight, a->weight, a->bias, a->gate, a->scale, a->shift};
  if (!aligned(a->x, xs) || !aligned(a->residual, rs) || !aligned(a->residual_out, rs)) return MXFP4_ERR_UNSUPPORTED;
  for (const void* v : vecs)
    if (!aligned(v, vs)) return MXFP4_ERR_UNSUPPORTED;

  // the vector path: 16-byte chunks of 8 columns
  bool vec = a->d % 8 == 0 && aligned(a->x, 16) && (a->ld_x * xs) % 16 == 0 && aligned(a->residual, 16) &&
             aligned(a->residual_out, 16);
  if (a->residual != nullptr) vec = vec && (a->ld_r * rs) % 16 == 0;
  if (a->residual_out != nullptr) vec = vec && (a->ld_ro * rs) % 16 == 0;
  if (grouped) vec = vec && (a->ld_vec * vs) % 16 == 0;
  for (const void* v : vecs) vec = vec && aligned(v, 16);
  if (!dense && !vec) return MXFP4_ERR_UNSUPPORTED;

  k.x = a->x;
  k.residual = a->residual;
  k.residual_out = a->residual_out;
  k.post_weight = a->post_weight;
  k.weight = a->weight;
  k.bias = a->bias;
  k.gate = a->gate;
  k.scale = a->scale;
  k.shift = a->shift;
  k.ld_x = a->ld_x;
  k.ld_r = a->ld_r;
  k.ld_ro = a->ld_ro;
  k.ld_vec = a->ld_vec;
  k.rows = static_cast<uint32_t>(a->rows);
  k.d = static_cast<uint32_t>(a->d);
  k.group_rows = !grouped || a->group_rows >= a->rows ? k.rows : static_cast<uint32_t>(a->group_rows);
  k.x_bf16 = a->x_dtype == MXFP4_BF16;
  k.r_bf16 = a->r_dtype == MXFP4_BF16;
  k.vec_bf16 = a->vec_dtype == MXFP4_BF16;
  k.layer = a->kind == MXFP4_NORM_LAYER;
  k.post_norm = a->post_norm != 0;
  k.vec = vec;
  k.residual_scale = a->residual_scale;
  k.eps = a->eps;
  return MXFP4_OK;
}

// The checks that the GEMMs with an epilogue share: sizes, operands (a second
// weight for the gated form) and limits; then g's operands.
mxfp4_status parse_operands(const uint8_t* a_codes, const uint8_t* a_scales, int64_t m, const uint8_t* b_codes,
                            const uint8_t* b_scales, const uint8_t* u_codes, const uint8_t* u_scales, bool glu,
                            int64_t n, int64_t k, bool tiled, mxfp4::FusedArgs& f) {
  if (a_codes == nullptr || a_scales == nullptr || b_codes == nullptr || b_scales == nullptr) return MXFP4_ERR_INVALID_ARG;
  if (glu && (u_codes == nullptr || u_scales == nullptr)) return MXFP4_ERR_INVALID_ARG;
  if (m >= kMaxDim || n >= kMaxDim || k >= kMaxDim) return MXFP4_ERR_UNSUPPORTED;
  if (!aligned(a_codes, 16) || !aligned(b_codes, 16) || !aligned(u_codes, 16)) return MXFP4_ERR_UNSUPPORTED;
  if (tiled && (!aligned(a_scales, 4) || !aligned(b_scales, 4) || !aligned(u_scales, 4))) return MXFP4_ERR_UNSUPPORTED;
  f.g.a_codes = a_codes;
  f.g.a_scales = a_scales;
  f.g.b_codes = b_codes;
  f.g.b_scales = b_scales;
  f.g.m = static_cast<int32_t>(m);
  f.g.n = static_cast<int32_t>(n);
  f.g.k = static_cast<int32_t>(k);
  f.g.tiled = tiled;
  f.glu = glu;
  f.u_codes = u_codes;
  f.u_scales = u_scales;
  return MXFP4_OK;
}

mxfp4_status launch_fused(const mxfp4::FusedArgs& f, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  switch (mxfp4::fused_route(f)) {
    case mxfp4::FusedRoute::kSmall: return from_hip(mxfp4::launch_fused_small(f, s));
    case mxfp4::FusedRoute::kMid: return from_hip(mxfp4::launch_fused_tiles(f, true, s));
    case mxfp4::FusedRoute::kLarge: return from_hip(mxfp4::launch_fused_tiles(f, false, s));
    default: return MXFP4_ERR_UNSUPPORTED;
  }
}

// act, the vectors and their types of an epilogue (NULL: none)
mxfp4_status check_epilogue(const mxfp4_epilogue* e, int64_t n) {
  if (e == nullptr) return MXFP4_OK;
  if (!is_act(e->act) || !is_dtype(e->vec_dtype) || !is_dtype(e->res_dtype) || e->reserved != 0)
    return MXFP4_ERR_INVALID_ARG;
  if (e->gate != nullptr && (e->ld_gate < n || e->group_rows < 1)) return MXFP4_ERR_INVALID_ARG;
  if (e->residual != nullptr && e->ld_res < n) return MXFP4_ERR_INVALID_ARG;
  return MXFP4_OK;
}

mxfp4_status set_epilogue(const mxfp4_epilogue* e, mxfp4::FusedArgs& f) {
  if (e == nullptr) return MXFP4_OK;
  const int64_t vs = size_of(e->vec_dtype);
  if (!aligned(e->bias, vs) || !aligned(e->gate, vs) || !aligned(e->residual, size_of(e->res_dtype)))
    return MXFP4_ERR_UNSUPPORTED;
  f.act = e->act;
  f.vec_bf16 = e->vec_dtype == MXFP4_BF16;
  f.bias = e->bias;
  f.gate = e->gate;
  f.ld_gate = e->ld_gate;
  // one group where a group holds every row
  f.group_rows = e->gate == nullptr || e->group_rows >= f.g.m ? static_cast<uint32_t>(f.g.m)
                                                              : static_cast<uint32_t>(e->group_rows);
  f.residual = e->residual;
  f.ld_res = e->ld_res;
  f.res_bf16 = e->res_dtype == MXFP4_BF16;
  return MXFP4_OK;
}

mxfp4_status check_glu(const mxfp4_glu* w) {
  if (w == nullptr || !is_act(w->act) || !is_dtype(w->vec_dtype) || w->reserved != 0) return MXFP4_ERR_INVALID_ARG;
  return MXFP4_OK;
}

mxfp4_status set_glu(const mxfp4_glu* w, mxfp4::FusedArgs& f) {
  const int64_t vs = size_of(w->vec_dtype);
  if (!aligned(w->bias_g, vs) || !aligned(w->bias_u, vs)) return MXFP4_ERR_UNSUPPORTED;
  f.act = w->act;
  f.vec_bf16 = w->vec_dtype == MXFP4_BF16;
  f.bias = w->bias_g;
  f.bias_u = w->bias_u;
  return MXFP4_OK;
}

}  // namespace

extern "C" {

MXFP4_API mxfp4_status mxfp4_norm(const mxfp4_norm_args* a, void* y, int32_t y_dtype, int64_t ld_y, void* stream) {
  mxfp4::NormArgs k{};
  const mxfp4_status st = parse_norm(a, true, k);
  if (st != MXFP4_OK) return st;
  if (!is_dtype(y_dtype) || (y != nullptr && ld_y < a->d)) return MXFP4_ERR_INVALID_ARG;
  if (a->rows == 0) return MXFP4_OK;
  if (y == nullptr && a->residual_out == nullptr) return MXFP4_ERR_INVALID_ARG;
  if (!aligned(y, size_of(y_dtype))) return MXFP4_ERR_UNSUPPORTED;
  k.y = y;
  k.ld_y = ld_y;
  k.y_bf16 = y_dtype == MXFP4_BF16;
  if (y != nullptr) k.vec = k.vec && aligned(y, 16) && (ld_y * size_of(y_dtype)) % 16 == 0;
  return from_hip(mxfp4::launch_norm(k, static_cast<hipStream_t>(stream)));
}

MXFP4_API mxfp4_status mxfp4_norm_quantize(const mxfp4_norm_args* a, const mxfp4_rotation* rot, int32_t layout,
                                           uint8_t* codes, uint8_t* scales, void* stream) {
  if (!is_layout(layout)) return MXFP4_ERR_INVALID_ARG;
  const bool tiled = layout == MXFP4_LAYOUT_TILED;
  Rot r;
  const mxfp4_status rs = parse_rotation(rot, r);
  if (rs != MXFP4_OK) return rs;
  if (a != nullptr && a->d >= 1 && (a->d % (tiled ? mxfp4::kTileK : 32)) != 0) return MXFP4_ERR_INVALID_ARG;
  mxfp4::NormArgs k{};
  const mxfp4_status st = parse_norm(a, false, k);
  if (st != MXFP4_OK) return st;
  if (a->rows == 0) return MXFP4_OK;
  if (codes == nullptr || scales == nullptr) return MXFP4_ERR_INVALID_ARG;
  if (!aligned(codes, 16) || (tiled && !aligned(scales, 4))) return MXFP4_ERR_UNSUPPORTED;
  if (r.kind == MXFP4_ROT_KRON && a->d > mxfp4::kNormMaxDKron) return MXFP4_ERR_UNSUPPORTED;
  const int64_t rows_pad = tiled ? (a->rows + mxfp4::kTileRows - 1) / mxfp4::kTileRows * mxfp4::kTileRows : a->rows;
  if (rows_pad * (a->d / 32) >= (int64_t(1) << 31)) return MXFP4_ERR_UNSUPPORTED;
  k.codes = codes;
  k.scales = scales;
  k.tiled = tiled;
  k.rot = r.kind;
  k.p = r.p;
  k.q = r.q;
  k.fa = r.fa;
  k.fb = r.fb;
  return from_hip(mxfp4::launch_norm(k, static_cast<hipStream_t>(stream)));
}

MXFP4_API mxfp4_status mxfp4_gemm_epilogue(const uint8_t* a_codes, const uint8_t* a_scales, int64_t m,
                                           const uint8_t* b_codes, const uint8_t* b_scales, int64_t n, int64_t k,
                                           int32_t layout, const mxfp4_epilogue* e, void* y, int32_t y_dtype,
                                           int64_t ld_y, void* stream) {
  if (!is_dtype(y_dtype) || !is_layout(layout) || !sizes_ok(m, n, k, layout) || ld_y < n) return MXFP4_ERR_INVALID_ARG;
  mxfp4_status st = check_epilogue(e, n);
  if (st != MXFP4_OK) return st;
  if (m == 0 || n == 0) return MXFP4_OK;
  mxfp4::FusedArgs f;
  st = parse_operands(a_codes, a_scales, m, b_codes, b_scales, nullptr, nullptr, false, n, k,
                      layout == MXFP4_LAYOUT_TILED, f);
  if (st == MXFP4_OK) st = dense_output(y, y_dtype, ld_y, f);
  if (st == MXFP4_OK) st = set_epilogue(e, f);
  return st == MXFP4_OK ? launch_fused(f, stream) : st;
}

MXFP4_API mxfp4_status mxfp4_gemm_epilogue_requant(const uint8_t* a_codes, const uint8_t* a_scales, int64_t m,
                                                   const uint8_t* b_codes, const uint8_t* b_scales, int64_t n,
                                                   int64_t k, int32_t layout, const mxfp4_epilogue* e,
                                                   const mxfp4_rotation* rot, uint8_t* y_codes, uint8_t* y_scales,
                                                   int32_t y_layout, void* stream) {
  if (!is_layout(layout) || !is_layout(y_layout) || !sizes_ok(m, n, k, layout)) return MXFP4_ERR_INVALID_ARG;
  Rot r;
  mxfp4_status st = parse_rotation(rot, r);
  if (st == MXFP4_OK) st = check_epilogue(e, n);
  if (st != MXFP4_OK) return st;
  if (m == 0 || n == 0) return MXFP4_OK;
  mxfp4::FusedArgs f;
  st = parse_operands(a_codes, a_scales, m, b_codes, b_scales, nullptr, nullptr, false, n, k,
                      layout == MXFP4_LAYOUT_TILED, f);
  if (st == MXFP4_OK) st = packed_output(r, y_codes, y_scales, y_layout, n, f);
  if (st == MXFP4_OK && e != nullptr && (e->gate != nullptr || e->residual != nullptr)) st = MXFP4_ERR_UNSUPPORTED;
  if (st == MXFP4_OK) st = set_epilogue(e, f);
  return st == MXFP4_OK ? launch_fused(f, stream) : st;
}

MXFP4_API mxfp4_status mxfp4_gemm_glu(const uint8_t* a_codes, const uint8_t* a_scales, int64_t m, const mxfp4_glu* w,
                                      int64_t n, int64_t k, int32_t layout, void* y, int32_t y_dtype, int64_t ld_y,
                                      void* stream) {
  if (!is_dtype(y_dtype) || !is_layout(layout) || !sizes_ok(m, n, k, layout) || ld_y < n) return MXFP4_ERR_INVALID_ARG;
  mxfp4_status st = check_glu(w);
  if (st != MXFP4_OK) return st;
  if (m == 0 || n == 0) return MXFP4_OK;
  mxfp4::FusedArgs f;
  st = parse_operands(a_codes, a_scales, m, w->g_codes, w->g_scales, w->u_codes, w->u_scales, true, n, k,
                      layout == MXFP4_LAYOUT_TILED, f);
  if (st == MXFP4_OK) st = dense_output(y, y_dtype, ld_y, f);
  if (st == MXFP4_OK) st = set_glu(w, f);
  return st == MXFP4_OK ? launch_fused(f, stream) : st;
}

MXFP4_API mxfp4_status mxfp4_gemm_glu_requant(const uint8_t* a_codes, const uint8_t* a_scales, int64_t m,
                                              const mxfp4_glu* w, int64_t n, int64_t k, int32_t layout,
                                              const mxfp4_rotation* rot, uint8_t* y_codes, uint8_t* y_scales,
                                              int32_t y_layout, void* stream) {
  if (!is_layout(layout) || !is_layout(y_layout) || !sizes_ok(m, n, k, layout)) return MXFP4_ERR_INVALID_ARG;
  Rot r;
  mxfp4_status st = parse_rotation(rot, r);
  if (st == MXFP4_OK) st = check_glu(w);
  if (st != MXFP4_OK) return st;
  if (m == 0 || n == 0) return MXFP4_OK;
  mxfp4::FusedArgs f;
  st = parse_operands(a_codes, a_scales, m, w->g_codes, w->g_scales, w->u_codes, w->u_scales, true, n, k,
                      layout == MXFP4_LAYOUT_TILED, f);
  if (st == MXFP4_OK) st = packed_output(r, y_codes, y_scales, y_layout, n, f);
  if (st == MXFP4_OK) st = set_glu(w, f);
  return st == MXFP4_OK ? launch_fused(f, stream) : st;
}

}  // extern "C"
