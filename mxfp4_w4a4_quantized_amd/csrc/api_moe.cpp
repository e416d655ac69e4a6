// C-ABI of the mixture-of-experts operators: argument validation, kernel
// selection, HIP error mapping.  The declarations and error behaviour are
// documented in mxfp4.h.
#include "mxfp4.h"

#include <cmath>
#include <cstdint>

#include "args.h"
#include "moe_plan.h"

using namespace mxfp4::args;

namespace {

constexpr int kMaxTopk = 64;

// Sizes that a plan is made of.
mxfp4_status check_plan_sizes(int64_t tokens, int64_t topk, int64_t experts) {
  if (tokens < 0 || topk < 1 || experts < 1) return MXFP4_ERR_INVALID_ARG;
  if (topk > kMaxTopk || experts > mxfp4::moe::kMaxExperts || tokens >= mxfp4::moe::kMaxPairs / topk)
    return MXFP4_ERR_UNSUPPORTED;
  return MXFP4_OK;
}

// The experts that the tokens are spread over: the plan's where none are given.
mxfp4_status check_spread(int32_t router_experts, int64_t experts) {
  if (router_experts != 0 && router_experts < experts) return MXFP4_ERR_INVALID_ARG;
  return router_experts > mxfp4::moe::kMaxExperts ? MXFP4_ERR_UNSUPPORTED : MXFP4_OK;
}

// The plan's part of a product's arguments.
void set_plan(const void* plan, int64_t pairs, int64_t experts, int32_t router_experts, mxfp4::MoeArgs& f) {
  const mxfp4::moe::PlanLayout l = mxfp4::moe::plan_layout(pairs, experts);
  const int32_t* p = static_cast<const int32_t*>(plan);
  for (int i = 0; i < mxfp4::moe::kHeights; ++i) f.tiles[i] = p + l.tiles[i];
  f.ntiles = p + l.ntiles;
  f.experts = static_cast<int32_t>(experts);
  f.spread = router_experts != 0 ? router_experts : f.experts;
}

// The height of a product's row tiles.  The tile kernels hold 32-bit offsets within A
// (`rows` rows) and within one expert's weights, and 32-bit tile numbers: past those
// few rows an expert go in tiles of 16, many are refused.
mxfp4_status choose_height(const mxfp4::MoeArgs& f, int64_t rows, int& height) {
  height = mxfp4::moe_tile_rows(f);
  if (height < 128) return MXFP4_OK;
  const int64_t n = f.g.n, k = f.g.k, arows = (rows + mxfp4::kTileRows - 1) / mxfp4::kTileRows * mxfp4::kTileRows;
  const int64_t limit = int64_t(1) << 32, tiles_n = (n + 63) / 64;
  if (arows * (k / 2) < limit && (n + 255) / 256 * 256 * (k / 2) < limit &&
      mxfp4::moe::max_tiles(f.g.m, f.experts, height) * tiles_n < (int64_t(1) << 31))
    return MXFP4_OK;
  height = 16;
  return f.g.m / f.spread <= 18 ? MXFP4_OK : MXFP4_ERR_UNSUPPORTED;
}

// Operands of a product: `rows` rows of A, `pairs` of the result, experts' weights
// of n x k.  Then the kernel: its row tiles' height.
mxfp4_status set_operands(const uint8_t* a_codes, const uint8_t* a_scales, int64_t rows, int64_t pairs,
                          const uint8_t* w_codes, const uint8_t* w_scales, const uint8_t* g_codes,
                          const uint8_t* g_scales, bool glu, int64_t n, int64_t k, int32_t layout, mxfp4::MoeArgs& f,
                          int& height) {
  if (a_codes == nullptr || a_scales == nullptr || w_codes == nullptr || w_scales == nullptr) return MXFP4_ERR_INVALID_ARG;
  if (glu && (g_codes == nullptr || g_scales == nullptr)) return MXFP4_ERR_INVALID_ARG;
  if (n >= kMaxDim || k >= kMaxDim) return MXFP4_ERR_UNSUPPORTED;
  if (!aligned(a_codes, 16) || !aligned(w_codes, 16) || !aligned(g_codes, 16)) return MXFP4_ERR_UNSUPPORTED;
  const bool tiled = layout == MXFP4_LAYOUT_TILED;
  if (k % mxfp4::kTileK == 0 && (!aligned(a_scales, 4) || !aligned(w_scales, 4) || !aligned(g_scales, 4)))
    return MXFP4_ERR_UNSUPPORTED;
  const int64_t wrows = tiled ? (n + mxfp4::kTileRows - 1) / mxfp4::kTileRows * mxfp4::kTileRows : n;
  f.g.a_codes = a_codes;
  f.g.a_scales = a_scales;
  // (gated: the first weight is the gate projection)
  f.g.b_codes = glu ? g_codes : w_codes;
  f.g.b_scales = glu ? g_scales : w_scales;
  f.u_codes = glu ? w_codes : nullptr;
  f.u_scales = glu ? w_scales : nullptr;
  f.glu = glu;
  f.g.m = static_cast<int32_t>(pairs);
  f.g.n = static_cast<int32_t>(n);
  f.g.k = static_cast<int32_t>(k);
  f.g.tiled = tiled;
  f.a_rows = static_cast<int32_t>(rows);
  f.a_tiled = tiled;
  f.w_codes = wrows * (k / 2);
  f.w_scales = wrows * (k / 32);
  return choose_height(f, rows, height);
}

mxfp4_status launch(const mxfp4::MoeArgs& f, int height, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return from_hip(height < 128 ? mxfp4::launch_moe_small(f, height, s) : mxfp4::launch_moe_tiles(f, height == 128, s));
}

mxfp4_status check_up(const mxfp4_moe_up_weights* w) {
  if (w == nullptr || !is_act(w->act) || !is_dtype(w->vec_dtype)) return MXFP4_ERR_INVALID_ARG;
  if (w->g_codes == nullptr && (w->g_scales != nullptr || w->bias_g != nullptr)) return MXFP4_ERR_INVALID_ARG;
  return MXFP4_OK;
}

// The common part of moe_up and moe_up_requant, up to their outputs.
mxfp4_status parse_up(const uint8_t* a_codes, const uint8_t* a_scales, const void* plan, int64_t tokens, int64_t topk,
                      int64_t experts, const mxfp4_moe_up_weights* w, int64_t n, int64_t k, int32_t layout,
                      mxfp4::MoeArgs& f, int& height) {
  if (plan == nullptr) return MXFP4_ERR_INVALID_ARG;
  if (!aligned(plan, 16)) return MXFP4_ERR_UNSUPPORTED;
  const int64_t vs = size_of(w->vec_dtype);
  if (!aligned(w->bias_u, vs) || !aligned(w->bias_g, vs)) return MXFP4_ERR_UNSUPPORTED;
  set_plan(plan, tokens * topk, experts, w->router_experts, f);
  const bool glu = w->g_codes != nullptr;
  const mxfp4_status st = set_operands(a_codes, a_scales, tokens, tokens * topk, w->u_codes, w->u_scales, w->g_codes,
                                       w->g_scales, glu, n, k, layout, f, height);
  if (st != MXFP4_OK) return st;
  f.token = static_cast<const int32_t*>(plan) + mxfp4::moe::plan_layout(tokens * topk, experts).token;
  f.act = w->act;
  f.vec_bf16 = w->vec_dtype == MXFP4_BF16;
  f.bias = glu ? w->bias_g : w->bias_u;
  f.bias_u = glu ? w->bias_u : nullptr;
  return MXFP4_OK;
}

// Where moe_down's products go before the sum: 16-bit values with a power of two
// per 32 columns (tile kernels, bf16 results), or fp32.
bool half_products(const mxfp4::MoeArgs& f, int height, int32_t y_dtype) {
  return height >= 128 && y_dtype == MXFP4_BF16 && f.g.n % 32 == 0;
}
int64_t product_bytes(int64_t pairs, int64_t n, bool half) {
  const int64_t values = pairs * n * (half ? 2 : 4);
  return (values + 255) / 256 * 256 + (half ? pairs * (n / 32) : 0);
}

mxfp4_status check_down_sizes(int64_t tokens, int64_t topk, int64_t experts, int64_t n, int64_t k, int32_t layout,
                              int32_t y_dtype) {
  if (!is_layout(layout) || !is_dtype(y_dtype) || !sizes_ok(tokens, n, k, layout)) return MXFP4_ERR_INVALID_ARG;
  const mxfp4_status st = check_plan_sizes(tokens, topk, experts);
  if (st != MXFP4_OK) return st;
  return n >= kMaxDim || k >= kMaxDim ? MXFP4_ERR_UNSUPPORTED : MXFP4_OK;
}

}  // namespace

extern "C" {

MXFP4_API mxfp4_status mxfp4_moe_route(const void* logits, int32_t dtype, int64_t tokens, int64_t experts, int64_t ld,
                                       const mxfp4_router* r, int32_t* ids, float* weights, void* stream) {
  if (r == nullptr || r->reserved != 0 || !is_dtype(dtype)) return MXFP4_ERR_INVALID_ARG;
  if (r->score != MXFP4_SCORE_SOFTMAX && r->score != MXFP4_SCORE_SIGMOID) return MXFP4_ERR_INVALID_ARG;
  if (r->group_score != MXFP4_GROUP_MAX && r->group_score != MXFP4_GROUP_TOP2) return MXFP4_ERR_INVALID_ARG;
  if (tokens < 0 || experts < 1 || ld < experts || r->topk < 1 || r->topk > experts) return MXFP4_ERR_INVALID_ARG;
  if (r->groups < 1 || experts % r->groups != 0 || r->topk_groups < 1 || r->topk_groups > r->groups) return MXFP4_ERR_INVALID_ARG;
  if (!std::isfinite(r->scale)) return MXFP4_ERR_INVALID_ARG;
  if (experts > mxfp4::moe::kMaxExperts || r->topk > kMaxTopk || r->groups > 64 || tokens >= kMaxDim) return MXFP4_ERR_UNSUPPORTED;
  if (tokens == 0) return MXFP4_OK;
  if (logits == nullptr || ids == nullptr || weights == nullptr) return MXFP4_ERR_INVALID_ARG;
  if (!aligned(logits, size_of(dtype)) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(r->bias, 4)) return MXFP4_ERR_UNSUPPORTED;
  mxfp4::RouteArgs a{};
  a.logits = logits;
  a.bias = r->bias;
  a.ids = ids;
  a.weights = weights;
  a.tokens = tokens;
  a.ld = ld;
  a.experts = static_cast<int32_t>(experts);
  a.topk = r->topk;
  a.groups = r->groups;
  a.topk_groups = r->topk_groups;
  a.bf16 = dtype == MXFP4_BF16;
  a.softmax = r->score == MXFP4_SCORE_SOFTMAX;
  a.group_top2 = r->group_score == MXFP4_GROUP_TOP2;
  a.renormalize = r->renormalize != 0;
  a.scale = r->scale;
  return from_hip(mxfp4::launch_moe_route(a, static_cast<hipStream_t>(stream)));
}

MXFP4_API mxfp4_status mxfp4_moe_plan_bytes(int64_t tokens, int64_t topk, int64_t experts, int64_t* bytes) {
  if (bytes == nullptr) return MXFP4_ERR_INVALID_ARG;
  const mxfp4_status st = check_plan_sizes(tokens, topk, experts);
  if (st != MXFP4_OK) return st;
  *bytes = mxfp4::moe::plan_layout(tokens * topk, experts).words * 4;
  return MXFP4_OK;
}

MXFP4_API mxfp4_status mxfp4_moe_plan(const int32_t* ids, int64_t tokens, int64_t topk, int64_t first, int64_t experts,
                                      void* plan, int64_t plan_bytes, void* stream) {
  if (first < 0) return MXFP4_ERR_INVALID_ARG;
  const mxfp4_status st = check_plan_sizes(tokens, topk, experts);
  if (st != MXFP4_OK) return st;
  if (first >= kMaxDim) return MXFP4_ERR_UNSUPPORTED;
  const int64_t pairs = tokens * topk;
  const mxfp4::moe::PlanLayout l = mxfp4::moe::plan_layout(pairs, experts);
  if (plan == nullptr || plan_bytes < l.words * 4 || (pairs > 0 && ids == nullptr)) return MXFP4_ERR_INVALID_ARG;
  if (!aligned(plan, 16) || !aligned(ids, 4)) return MXFP4_ERR_UNSUPPORTED;
  int32_t* p = static_cast<int32_t*>(plan);
  mxfp4::PlanArgs a{};
  a.ids = ids;
  a.pairs = pairs;
  a.chunk = mxfp4::moe::chunk_pairs(pairs);
  a.topk = static_cast<int32_t>(topk);
  a.first = static_cast<int32_t>(first);
  a.experts = static_cast<int32_t>(experts);
  a.offsets = p;
  a.order = p + l.order;
  a.slot = p + l.slot;
  a.token = p + l.token;
  a.ntiles = p + l.ntiles;
  for (int i = 0; i < mxfp4::moe::kHeights; ++i) a.tiles[i] = p + l.tiles[i];
  a.counts = p + l.counts;
  return from_hip(mxfp4::launch_moe_plan(a, static_cast<hipStream_t>(stream)));
}

MXFP4_API mxfp4_status mxfp4_moe_up(const uint8_t* a_codes, const uint8_t* a_scales, const void* plan, int64_t tokens,
                                    int64_t topk, int64_t experts, const mxfp4_moe_up_weights* w, int64_t n, int64_t k,
                                    int32_t layout, void* y, int32_t y_dtype, int64_t ld_y, void* stream) {
  if (!is_dtype(y_dtype) || !is_layout(layout) || !sizes_ok(tokens, n, k, layout) || ld_y < n) return MXFP4_ERR_INVALID_ARG;
  mxfp4_status st = check_up(w);
  if (st == MXFP4_OK) st = check_plan_sizes(tokens, topk, experts);
  if (st == MXFP4_OK) st = check_spread(w->router_experts, experts);
  if (st != MXFP4_OK) return st;
  if (tokens == 0 || n == 0) return MXFP4_OK;
  mxfp4::MoeArgs f;
  int height = 0;
  st = parse_up(a_codes, a_scales, plan, tokens, topk, experts, w, n, k, layout, f, height);
  if (st == MXFP4_OK) st = dense_output(y, y_dtype, ld_y, f);
  return st == MXFP4_OK ? launch(f, height, stream) : st;
}

MXFP4_API mxfp4_status mxfp4_moe_up_requant(const uint8_t* a_codes, const uint8_t* a_scales, const void* plan,
                                            int64_t tokens, int64_t topk, int64_t experts,
                                            const mxfp4_moe_up_weights* w, int64_t n, int64_t k, int32_t layout,
                                            const mxfp4_rotation* rot, uint8_t* y_codes, uint8_t* y_scales,
                                            int32_t y_layout, void* stream) {
  if (!is_layout(layout) || !is_layout(y_layout) || !sizes_ok(tokens, n, k, layout)) return MXFP4_ERR_INVALID_ARG;
  Rot r;
  mxfp4_status st = parse_rotation(rot, r);
  if (st == MXFP4_OK) st = check_up(w);
  if (st == MXFP4_OK) st = check_plan_sizes(tokens, topk, experts);
  if (st == MXFP4_OK) st = check_spread(w->router_experts, experts);
  if (st != MXFP4_OK) return st;
  if (tokens == 0 || n == 0) return MXFP4_OK;
  mxfp4::MoeArgs f;
  int height = 0;
  st = parse_up(a_codes, a_scales, plan, tokens, topk, experts, w, n, k, layout, f, height);
  if (st == MXFP4_OK) st = packed_output(r, y_codes, y_scales, y_layout, n, f);
  return st == MXFP4_OK ? launch(f, height, stream) : st;
}

MXFP4_API mxfp4_status mxfp4_moe_down_workspace(int64_t tokens, int64_t topk, int64_t experts, int64_t n, int64_t k,
                                                int32_t layout, int32_t y_dtype, int64_t* bytes) {
  if (bytes == nullptr) return MXFP4_ERR_INVALID_ARG;
  mxfp4_status st = check_down_sizes(tokens, topk, experts, n, k, layout, y_dtype);
  if (st != MXFP4_OK) return st;
  mxfp4::MoeArgs f;
  f.g.m = static_cast<int32_t>(tokens * topk);
  f.g.n = static_cast<int32_t>(n);
  f.g.k = static_cast<int32_t>(k);
  f.experts = f.spread = static_cast<int32_t>(experts);
  f.g.tiled = layout == MXFP4_LAYOUT_TILED;
  int height = 0;
  if (tokens > 0 && n > 0) st = choose_height(f, f.g.m, height);
  if (st != MXFP4_OK) return st;
  *bytes = tokens == 0 || n == 0 || mxfp4::moe_down_small(f) ? 0 : product_bytes(tokens * topk, n, half_products(f, height, y_dtype));
  return MXFP4_OK;
}

MXFP4_API mxfp4_status mxfp4_moe_down(const uint8_t* h_codes, const uint8_t* h_scales, const void* plan, int64_t tokens,
                                      int64_t topk, int64_t experts, const float* weights,
                                      const mxfp4_moe_down_weights* w, int64_t n, int64_t k, int32_t layout,
                                      const void* residual, int32_t res_dtype, int64_t ld_res, void* y,
                                      int32_t y_dtype, int64_t ld_y, void* workspace, int64_t workspace_bytes,
                                      void* stream) {
  if (w == nullptr || !is_dtype(w->vec_dtype) || !is_dtype(res_dtype)) return MXFP4_ERR_INVALID_ARG;
  if (ld_y < n || (residual != nullptr && ld_res < n)) return MXFP4_ERR_INVALID_ARG;
  mxfp4_status st = check_down_sizes(tokens, topk, experts, n, k, layout, y_dtype);
  if (st == MXFP4_OK) st = check_spread(w->router_experts, experts);
  if (st != MXFP4_OK) return st;
  if (tokens == 0 || n == 0) return MXFP4_OK;
  if (plan == nullptr || weights == nullptr || y == nullptr) return MXFP4_ERR_INVALID_ARG;
  if (!aligned(plan, 16) || !aligned(weights, 4) || !aligned(y, size_of(y_dtype)) || !aligned(residual, size_of(res_dtype)) ||
      !aligned(w->bias, size_of(w->vec_dtype)))
    return MXFP4_ERR_UNSUPPORTED;
  const int64_t pairs = tokens * topk;
  mxfp4::MoeArgs f;
  int height = 0;
  set_plan(plan, pairs, experts, w->router_experts, f);
  st = set_operands(h_codes, h_scales, pairs, pairs, w->codes, w->scales, nullptr, nullptr, false, n, k, layout, f, height);
  if (st != MXFP4_OK) return st;
  f.vec_bf16 = w->vec_dtype == MXFP4_BF16;
  f.bias = w->bias;
  mxfp4::CombineArgs c{};
  c.slot = static_cast<const int32_t*>(plan) + mxfp4::moe::plan_layout(pairs, experts).slot;
  c.weights = weights;
  c.residual = residual;
  c.ld_res = ld_res;
  c.res_bf16 = res_dtype == MXFP4_BF16;
  c.y = y;
  c.ld_y = ld_y;
  c.y_bf16 = y_dtype == MXFP4_BF16;
  c.tokens = tokens;
  c.topk = static_cast<int32_t>(topk);
  c.n = static_cast<int32_t>(n);
  if (mxfp4::moe_down_small(f)) return from_hip(mxfp4::launch_moe_down_small(f, c, static_cast<hipStream_t>(stream)));
  const bool half = half_products(f, height, y_dtype);
  if (workspace == nullptr || workspace_bytes < product_bytes(pairs, n, half)) return MXFP4_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return MXFP4_ERR_UNSUPPORTED;
  f.g.y = workspace;
  f.g.ld_y = n;
  f.g.y_bf16 = false;
  f.z_half = half;
  f.z_scales = half ? static_cast<uint8_t*>(workspace) + (pairs * n * 2 + 255) / 256 * 256 : nullptr;
  c.z = workspace;
  c.z_scales = f.z_scales;
  c.half = half;
  st = launch(f, height, stream);
  if (st != MXFP4_OK) return st;
  return from_hip(mxfp4::launch_moe_combine(c, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
