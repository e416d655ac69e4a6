// Internal launch interface between the C-ABI layer (api.cpp) and the HIP
// kernels.  Arguments reaching these functions are already validated.
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>

namespace mxfp4 {

struct QuantArgs {
  const void* x;
  int64_t ld_x;        // elements
  uint32_t rows;
  uint32_t nblk_row;   // k / 32
  int32_t rot;         // mxfp4_rot_kind
  int32_t p, q;        // Kronecker factor sizes
  const float* fa;     // p x p (Kronecker), or k per-channel factors (smoothing)
  const float* fb;     // q x q
  bool fit;            // fitted block exponents instead of the E8M0 rule
  uint8_t* codes;
  uint8_t* scales;
  bool tiled;          // MXFP4_LAYOUT_TILED outputs (nblk_row % 4 == 0)
  uint32_t rows_pad;   // rows rounded up to the 256-row tile (tiled only)
};

constexpr int kTileRows = 256;       // rows per tile of the tiled layout
constexpr int kTileK = 128;          // K elements per stage of the tiled layout

hipError_t launch_quantize(const QuantArgs& a, bool bf16, hipStream_t s);

struct GemmArgs {
  const uint8_t* a_codes;   // X side, m rows
  const uint8_t* a_scales;
  const uint8_t* b_codes;   // W side, n rows
  const uint8_t* b_scales;
  int32_t m, n, k;
  void* y;
  int64_t ld_y;
  bool y_bf16;
  bool tiled;               // both operands in MXFP4_LAYOUT_TILED
  // MXFP4 output (large-tile kernel only; n % 32 == 0, n % 128 == 0 when
  // q_tiled): Y requantized per 32-block along N into q_codes / q_scales
  // (y unused)
  bool q_out = false;
  bool q_tiled = false;     // output in MXFP4_LAYOUT_TILED
  uint8_t* q_codes = nullptr;
  uint8_t* q_scales = nullptr;
};

hipError_t launch_gemm(const GemmArgs& a, hipStream_t s);

// Compute units of the current device (cached per device; 256 if the query
// fails).
int cu_count();

// Large-tile persistent kernel (gemm_large.hip): K a multiple of 128,
// 4-byte aligned scale pointers, operand code bytes below 4 GiB; the only
// kernel for tiled operands.
bool gemm_large_supported(const GemmArgs& a);
hipError_t launch_gemm_large(const GemmArgs& a, hipStream_t s);
// Workgroups of the large-tile kernels for a number of output tiles.
int large_grid(int ntiles, int per_cu);

// Small-M kernel (gemm_small.hip): either layout; the kernel for decode
// shapes (m <= 64), bound by streaming the weights from HBM, and for shapes
// with fewer than 8 output tiles of 256 x 256 (gemm_small_route).
bool gemm_small_route(int64_t m, int64_t n);
bool gemm_small_supported(const GemmArgs& a);
hipError_t launch_gemm_small(const GemmArgs& a, hipStream_t s);

// Fused small-M linear layer (gemm_small.hip): the activations are rotated
// and quantized inside the GEMM kernel, in the same launch (1 <= m <= 64; W
// in either layout, described by g.b_* / g.tiled; g.a_* unused).
struct LinearArgs {
  const void* x;       // [m][ld_x] fp32 or bf16
  int64_t ld_x;        // elements
  bool x_bf16;
  int32_t rot;         // mxfp4_rot_kind
  int32_t p, q;
  const float* fa;
  const float* fb;
  GemmArgs g;
  // workspace: handoff counters (zero between calls) and the quantized
  // activations in MFMA operand order
  uint32_t* counters = nullptr;
  uint8_t* xq = nullptr;
};
bool linear_small_supported(const LinearArgs& a);
hipError_t launch_linear_small(const LinearArgs& a, hipStream_t s);
// Workspace of the fused layer: a fixed region of counters (the same for
// every shape, so one workspace serves calls of any shape), then the
// quantized activations, 1152 bytes per 16 rows and 128 K elements.
constexpr int64_t kLinearCounterBytes = 4096;
int64_t linear_small_workspace_bytes(int64_t m, int64_t k);
// The fixed scratch of the allocation-free variant: its device address on
// the current device (looked up, and its counters cleared on `s`, on the
// first call per device).
constexpr int64_t kLinearStaticScratchBytes = int64_t(4) << 20;
hipError_t linear_small_static_scratch(void** ptr, hipStream_t s);

// GEMM with a feed-forward epilogue (gemm_fused_small.hip,
// gemm_fused_large.hip): Y = residual + gate[g] * act(A B^T + bias), or, with
// glu, H = act(A B^T + bias) * (A U^T + bias_u); dense (g.y) or MXFP4 (g.q_*,
// after an optional Hadamard-32 along N; no gate or residual then).
struct FusedArgs {
  GemmArgs g;
  bool glu = false;
  const uint8_t* u_codes = nullptr;   // second weight, n rows, same layout
  const uint8_t* u_scales = nullptr;
  int32_t act = 0;                    // mxfp4_act
  bool vec_bf16 = false;              // type of the vectors below
  const void* bias = nullptr;         // n
  const void* bias_u = nullptr;       // n
  const void* gate = nullptr;         // [groups][ld_gate]
  int64_t ld_gate = 0;
  uint32_t group_rows = 1;            // rows of Y per gate row
  const void* residual = nullptr;     // [m][ld_res]
  int64_t ld_res = 0;
  bool res_bf16 = false;
  bool h32 = false;
};

// The kernel for a call: small-M, 128 x 128 or 256 x 256 tiles, or none.
enum class FusedRoute { kSmall, kMid, kLarge, kNone };
FusedRoute fused_route(const FusedArgs& a);
hipError_t launch_fused_small(const FusedArgs& a, hipStream_t s);
hipError_t launch_fused_tiles(const FusedArgs& a, bool mid, hipStream_t s);
hipError_t launch_glu_tiles(const FusedArgs& a, bool mid, hipStream_t s);        // its gated part
hipError_t launch_residual_tiles(const FusedArgs& a, bool mid, hipStream_t s);   // and that with a gate or a residual

// Experts' products (moe_small.hip, moe_tiles.hip): the rows of expert e, as a
// plan (moe_plan.h) orders them, by weight e of a stack.  g.m rows in all; row p
// of the result is that of plan row p.
struct MoeArgs : FusedArgs {
  const int32_t* tiles[4] = {};       // the plan's tile tables and their lengths
  const int32_t* ntiles = nullptr;    // [4]
  const int32_t* token = nullptr;     // row p reads row token[p] of A; null: row p
  int32_t a_rows = 0;                 // rows of A
  bool a_tiled = false;               // A's layout (g.tiled: the weights')
  int32_t experts = 0;
  int32_t spread = 0;                 // experts that the rows are spread over: those, or more on other GPUs
  int64_t w_codes = 0, w_scales = 0;  // bytes from one expert's weights to the next's
  // the result as 16-bit values with a power of two per 32 columns (g.y, z_scales)
  bool z_half = false;
  uint8_t* z_scales = nullptr;
};

// Norm with residual, gate and modulation (norm.hip); dense or MXFP4 result.
struct NormArgs {
  const void* x;
  const void* residual;
  void* residual_out;
  const void *post_weight, *weight, *bias;    // d
  const void *gate, *scale, *shift;           // [groups][ld_vec]
  int64_t ld_x, ld_r, ld_ro, ld_vec;
  uint32_t rows, d, group_rows;
  uint32_t row0 = 0;                          // first row of the launch
  bool x_bf16, r_bf16, vec_bf16;
  bool layer, post_norm;
  bool vec;                                   // every pointer and stride 16-byte aligned, d % 8 == 0
  float residual_scale, eps;
  // dense result (may be null)
  void* y = nullptr;
  int64_t ld_y = 0;
  bool y_bf16 = false;
  // MXFP4 result (may be null)
  uint8_t* codes = nullptr;
  uint8_t* scales = nullptr;
  bool tiled = false;
  int32_t rot = 0, p = 0, q = 0;              // mxfp4_rot_kind and its factors
  const float* fa = nullptr;
  const float* fb = nullptr;
};

constexpr int64_t kNormMaxD = 65536;          // row length
constexpr int64_t kNormMaxDKron = 16384;      // and with KRON, whose rows pass through LDS
hipError_t launch_norm(const NormArgs& a, hipStream_t s);

// Mixture of experts (moe_route.hip): router, plan and the weighted sum over a
// token's choices.
struct RouteArgs {
  const void* logits;    // [tokens][ld]
  const float* bias;     // [experts] or null
  int32_t* ids;          // [tokens][topk]
  float* weights;
  int64_t tokens, ld;
  int32_t experts, topk, groups, topk_groups;
  bool bf16, softmax, group_top2, renormalize;
  float scale;
};
hipError_t launch_moe_route(const RouteArgs& a, hipStream_t s);

struct PlanArgs {
  const int32_t* ids;    // [pairs]
  int64_t pairs, chunk;
  int32_t topk, first, experts;
  int32_t *offsets, *order, *slot, *token, *ntiles, *tiles[4], *counts;
};
hipError_t launch_moe_plan(const PlanArgs& a, hipStream_t s);

struct CombineArgs {
  const void* z;             // [rows][n] fp32, or 16-bit values with z_scales
  const uint8_t* z_scales;
  bool half;
  const int32_t* slot;       // [tokens][topk]
  const float* weights;
  const void* residual;      // [tokens][ld_res] or null
  int64_t ld_res;
  bool res_bf16;
  void* y;                   // [tokens][ld_y]
  int64_t ld_y;
  bool y_bf16;
  int64_t tokens;
  int32_t topk, n;
};
hipError_t launch_moe_combine(const CombineArgs& a, hipStream_t s);

// The kernel for the experts' products: row tiles of 16 or 32 (small-M), 128 or
// 256 rows.
int moe_tile_rows(const MoeArgs& f);
hipError_t launch_moe_small(const MoeArgs& f, int rows, hipStream_t s);
hipError_t launch_moe_tiles(const MoeArgs& f, bool mid, hipStream_t s);
// The down projection and the weighted sum in one kernel, and whether it is the one.
bool moe_down_small(const MoeArgs& f);
hipError_t launch_moe_down_small(const MoeArgs& f, const CombineArgs& c, hipStream_t s);

}  // namespace mxfp4
