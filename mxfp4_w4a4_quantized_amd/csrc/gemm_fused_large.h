// Large-tile MXFP4 GEMMs with a feed-forward epilogue, and their gated form:
//   Y = residual + gate[g] * act(A B^T + bias)
//   H = act(A G^T + bias) * (A U^T + bias_u)
// dense, or requantized to MXFP4 along N after an optional Hadamard-32.
//
// The main loop is gemm_large.hip's (its header describes it): persistent
// 4-wave workgroups on 256 x 256 tiles, a 4-stage LDS ring of direct loads that
// runs across tile boundaries, 128 x 128 accumulators per wave.  What differs:
//  * Bias.  It is added to the finished sums, so that a bias far above them
//    costs one rounding and not one per K step, and on the matrix pipe: one
//    v_mfma_f32_32x32x2_f32 per fragment, bias values of the fragment's 32
//    weight rows (K index 0) against ones, adds bias[row] to all 16 registers.
//    It runs one fragment ahead of the epilogue's vector work.  An fp32 MFMA
//    still holds that up for its 64 cycles (57344 x 3072 -> 12288, tanh GELU:
//    23 us in 1255), so the accumulators are cleared by a bf16 one, which does
//    not (their start from the bias, by an fp32 MFMA too, took as long as now:
//    1271 and 1275 us).
//  * Gated form.  A tile is 256 weight rows that alternate 32 rows of G and the
//    matching 32 rows of U, so a wave's even fragments hold the gate's
//    pre-activations and the odd ones the up projection's, for the same
//    outputs in the same lanes and registers: the product needs no exchange
//    and both weights keep their own layout (the ring's load plan picks the
//    rows).  128 output columns per tile.
//  * Epilogue.  Fragments leave the accumulators one at a time; act runs on the
//    16 values in registers.  bf16 and fp32 tiles are staged through the free
//    ring slot into whole row segments.  With a gate or a residual the staging
//    is fp32, so that act(x) is not rounded before them, and the finishing
//    lane holds 4 consecutive columns of one row: it reads the residual with
//    8- or 16-byte loads, issued a pass ahead.  MXFP4 tiles are requantized
//    from the registers.
//
// Bound by the matrix pipe at the clock the power limit leaves, then by the
// epilogue, during which a CU's only 256 x 256 tile feeds no MFMA.  Measured
// (bf16, H32 where MXFP4; the GEMM without an epilogue in brackets):
//  * 57344 x 3072 -> 12288, bias, tanh GELU   1171-1278 us, 3.4-3.7 PF/s (1018)
//  * 8192 x 4096 -> 2 x 14336, gated silu      455-477 us, 4.0-4.2 PF/s (434)
//  * 3584 x 12288 -> 3072, bias, gate, residual 79-84 us, 3.2-3.4 PF/s (69.5)
//  * 3584 x 3072 -> 12288, tanh GELU, H32, MXFP4  91-100 us, 2.7-3.0 PF/s (72.6)
//  * 523 x 1408 -> 2 x 3001 fp32, gated, bias      12-13 us (128 x 128 tiles)
//  * experts' products (MoeArgs): 8192 tokens x 8 of 64 experts, 4096 -> 2 x 2048,
//    gated silu, 620-650 us, 3.4-3.55 PF/s (65536 rows of one expert 542, of 64
//    experts with 1024 rows each in token order 585); 301 x 3 of 10, 1184 -> 2 x 1000
//    fp32, bias, 12.3 us (a tail of K)
// (over the cards; within a card to 1%.)
#pragma once
#include "gemm_large_core.h"
#include "activation.h"
#include "moe_tile.h"

#include <type_traits>
#include <utility>

namespace mxfp4 {
namespace large {

// A workgroup's output tile: TBN weight rows x TBM activation rows on 2 x 2
// waves, a ring of TNBUF stages, TWGS workgroups per CU.  TTAIL: row-major
// operands with K a multiple of 32 only.  The code blocks of the last stage past
// K are read as zeros, from a constant of their own; scale bytes, at addresses of
// any alignment, come one by one, a dword of LDS each.
template <int TBN, int TBM, int TNBUF, int TWGS, bool TTAIL = false>
struct Tile {
  static constexpr bool TAIL = TTAIL;
  static constexpr int BN = TBN, BM = TBM, NBUF = TNBUF, WGS = TWGS;
  static constexpr int WN = 2, WM = 2, NW = WN * WM, NT = 64 * NW;
  static constexpr int ROWS = BN + BM;                        // rows per stage: W then X
  static constexpr int CODE_BYTES = ROWS * RB;
  static constexpr int SCALE_BYTES = TAIL ? 16 : 4;           // per row
  static constexpr int STAGE_BYTES = CODE_BYTES + ROWS * SCALE_BYTES;
  static constexpr int FN = BN / WN / 32, FM = BM / WM / 32;  // 32 x 32 fragments per wave
  // Per stage and wave: code loads of 1 KiB (16 rows), in stage row order, and
  // scale loads of 64 rows (the last one repeated where they do not divide).
  static constexpr int CODE_LOADS = ROWS / 16 / NW, SCALE_LOADS = (ROWS / 64 + NW - 1) / NW;
  static constexpr int LPS = CODE_LOADS + SCALE_LOADS * (TAIL ? 4 : 1);
  static constexpr int CODE_LOADS_B = CODE_LOADS / 2;         // issued during sub-step 0
  static constexpr int NRD = FN + FM;                         // fragment reads per sub-step
  static constexpr int NRS = NRD * (TAIL ? 2 : 1);            // scale reads per stage
  static constexpr bool WHOLE = BN % (16 * CODE_LOADS) == 0;  // no wave loads rows of both sides
  static_assert(ROWS % (16 * NW) == 0 && BN % 64 == 0, "whole loads per wave and side");
  static_assert(TWGS * TNBUF * STAGE_BYTES <= 160 * 1024, "LDS ring exceeds 160 KiB");
};

// Direct global -> LDS loads of 16 and 4 bytes per lane.  (Functions of their
// own: inside a template that depends on the tile, the host pass drops the
// kernel's launch stub over the builtins.)
__device__ __forceinline__ void load_lds16(const uint8_t* src, uint8_t* dst) {
  __builtin_amdgcn_global_load_lds(src, dst, 16, 0, 0);
}
__device__ __forceinline__ void load_lds4(const uint8_t* src, uint8_t* dst) {
  __builtin_amdgcn_global_load_lds(src, dst, 4, 0, 0);
}
// A byte per lane, each zero-extended to a dword of LDS.
__device__ __forceinline__ void load_lds1(const uint8_t* src, uint8_t* dst) {
  __builtin_amdgcn_global_load_lds(src, dst, 1, 0, 0);
}
__device__ const uint4 kZeroBlock = {0, 0, 0, 0};

// Activation classes of the kernels that apply it in registers, to W values of a
// fragment at a time.
constexpr int A_LINEAR = 0;   // none or relu, by f.act
template <int ACT, int W>
__device__ __forceinline__ void activate(float (&v)[16], bool relu) {
  if constexpr (ACT == A_LINEAR) {
    if (relu) act::relu(v);
  } else if constexpr (ACT == act::GELU) {
    act::gelu(v);
  } else {
#pragma unroll
    for (int h = 0; h < 16; h += W) {
      float x[W];
#pragma unroll
      for (int r = 0; r < W; ++r) x[r] = v[h + r];
      if constexpr (ACT == act::SILU) act::silu(x);
      else act::gelu_tanh(x);
#pragma unroll
      for (int r = 0; r < W; ++r) v[h + r] = x[r];
    }
  }
}

// body(0), body(1), .. as straight-line code: the unroller gives up on a loop
// this long and would index the accumulators in scratch memory.
template <typename F, int... I>
__device__ __forceinline__ void each(F&& body, std::integer_sequence<int, I...>) {
  (body(std::integral_constant<int, I>{}), ...);
}

// acc = 0, by a product of zeros (bf16: two operand registers).  The s_nop and
// the wait states at the tile start are those of acc_zero_mfma.
__device__ __forceinline__ void acc_clear(v16f& acc, uint64_t zero) {
  asm volatile("s_nop 2\n\tv_mfma_f32_32x32x8_bf16 %0, %1, %1, 0" : "=a"(acc) : "v"(zero));
}

// acc[i][j] += bias of weight row i, for every j: one product and a zero, one
// rounding.  The compiler does not know it for an MFMA: the last MFMA before it
// that wrote acc, and the first read of acc after it, have to be 19 wait states
// (16 passes) away.
__device__ __forceinline__ void acc_add_bias(v16f& acc, float bias, float one) {
  asm volatile("s_nop 2\n\tv_mfma_f32_32x32x2_f32 %0, %1, %2, %0" : "+a"(acc) : "v"(bias), "v"(one));
}

__device__ __forceinline__ void mfma_wait() { asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory"); }

__device__ __forceinline__ float vec_elem(const void* p, bool bf16, int64_t i) {
  if (bf16) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  return static_cast<const float*>(p)[i];
}

// Hadamard-32 of a fragment's 32-block per row, in the quantizer's order: lane
// (row, g) holds column 8 t + 4 g + j in v[4 t + j].  Strides 1 and 2 run over
// j, 4 over the lane halves, 8 and 16 over t.  v_permlane32_swap turns the
// stride-4 butterflies of two registers into one add and one subtract of whole
// registers: [v0.lo v1.lo] +- [v0.hi v1.hi].  The halves stay swapped through
// the later strides, which treat every register alike.
__device__ __forceinline__ void swap_halves(float& a, float& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}

__device__ __forceinline__ void hadamard_fragment(float (&v)[16]) {
#pragma unroll
  for (int h = 1; h <= 2; h <<= 1)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (!(i & h)) {
        const float u = v[i], w = v[i + h];
        v[i] = u + w;
        v[i + h] = u - w;
      }
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    swap_halves(v[i], v[i + 1]);
    const float u = v[i], w = v[i + 1];
    v[i] = u + w;
    v[i + 1] = u - w;
  }
#pragma unroll
  for (int h = 4; h <= 8; h <<= 1)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (!(i & h)) {
        const float u = v[i], w = v[i + h];
        v[i] = u + w;
        v[i + h] = u - w;
      }
  const float c = __uint_as_float(0x3E3504F3u);   // nearest fp32 to 1/sqrt(32)
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = v[i] * c;
#pragma unroll
  for (int i = 0; i < 16; i += 2) swap_halves(v[i], v[i + 1]);
}

// Two fp32 -> packed 16-bit floats (low half = a), round to nearest even.
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, f16x2));
}

// Workgroups that a number of tiles is spread over, of `most`: the fewest (a
// multiple of 8) that need no more rounds, as large_grid does on the host.
__device__ __forceinline__ int balanced_grid(int ntiles, int most) {
  if (ntiles <= most) return ntiles;
  const int rounds = (ntiles + most - 1) / most;
  return min(most, ((ntiles + rounds - 1) / rounds + 7) / 8 * 8);
}

// ACT: A_LINEAR or an mxfp4_act.  OUT: 0 fp32, 1 bf16, 2 MXFP4.  RES: 0 no gate
// or residual; 1 / 2 a gate and/or a residual (bf16 / fp32) in whole aligned
// pieces of 4 columns, with at most two gate rows per wave; 3 any other.
//
// Args MoeArgs: the experts' products.  The tiles are those of the plan's row
// tiles, an expert's in one run (so that they share its weights in L2); how many
// there are is read from the plan, and workgroups without one leave.  A tile's
// weights are its expert's, its activation rows go by the plan's token numbers,
// a lane's 16 bytes of a row wherever the row lies.  OUT 3: 16-bit floats with a
// power of two per row and 32 columns.
template <class T, int ACT, int OUT, int RES, bool GLU, class Args = FusedArgs>
__global__ __launch_bounds__(T::NT, T::WGS) void gemm_fused_large_kernel(Args f, int tiles_m, int tiles_n, int grid,
                                                                 int xcd_remap) {
  constexpr bool MOE = std::is_same<Args, MoeArgs>::value;
  static_assert(RES == 0 || (OUT != 2 && !GLU), "gate and residual are for plain dense outputs");
  static_assert(!MOE || RES == 0, "no gate or residual in the experts' products");
  constexpr int BN = T::BN, BM = T::BM, NBUF = T::NBUF, WN = T::WN, WM = T::WM, NW = T::NW, FN = T::FN, FM = T::FM;
  constexpr int CODE_BYTES = T::CODE_BYTES, STAGE_BYTES = T::STAGE_BYTES, LPS = T::LPS, NRD = T::NRD;
  constexpr int CODE_LOADS = T::CODE_LOADS, SCALE_LOADS = T::SCALE_LOADS, CODE_LOADS_B = T::CODE_LOADS_B;
  constexpr int TN = GLU ? BN / 2 : BN;          // output columns per tile
  constexpr int WCOLS = TN / WN;                 // and per wave
  constexpr bool PIECES = RES == 1 || RES == 2;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[NBUF * STAGE_BYTES + (PIECES && FM * FN == 4 ? 1024 : 0)];

  const GemmArgs& g = f.g;
  constexpr int HI = moe::height_index(BM);
  if constexpr (MOE) {
    tiles_m = moe::uniform(f.ntiles + HI);
    grid = __builtin_amdgcn_readfirstlane(balanced_grid(tiles_m * tiles_n, grid));
    xcd_remap = (grid % 8) == 0;
    if ((int)blockIdx.x >= grid) return;
  }
  const int ntiles = tiles_m * tiles_n;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int b = blockIdx.x;
  const int slot = xcd_remap ? (b & 7) * (grid >> 3) + (b >> 3) : b;
  if (slot >= ntiles) return;
  const int nk = T::TAIL ? (g.k + KS - 1) / KS : g.k / KS;
  const int total = ((ntiles - slot + grid - 1) / grid) * nk;
  const uint32_t kbytes = (uint32_t)g.k / 2, kblocks = (uint32_t)g.k / 32;
  const int lr = lane & 31, lg = lane >> 5;

  // ---- direct LDS load plan, as gemm_large_kernel's: load i of a wave fills 16
  // stage rows (codes) or 64 (scales), weight rows first.  Gated: 32-row group
  // q of the weight side holds rows of G (q even) or U (q odd); a code load
  // takes 16 rows of one group, a scale load 64 rows (lanes 0-31 G, 32-63 U).
  const bool tiled = g.tiled;
  const uint32_t nstage = (uint32_t)nk;
  const bool w_first = CODE_LOADS * wave < BN / 16;   // this wave's first load: weight side
  auto code_group = [&](int i) { return CODE_LOADS * wave + i; };              // 16-row group of the stage
  auto code_w = [&](int i) { return T::WHOLE ? w_first : code_group(i) < BN / 16; };
  auto scale_group = [&](int i) { return min(SCALE_LOADS * wave + i, T::ROWS / 64 - 1); };
  auto scale_w = [&](int i) { return T::WHOLE ? w_first : scale_group(i) < BN / 64; };
  // The operands' addresses in registers, and selects between values (the
  // unary +): left to itself the compiler selects between the addresses of the
  // arguments, which puts a copy of them into scratch memory.
  auto held = [](const uint8_t* p) {
    uint64_t v = (uint64_t)p;
    asm("" : "+s"(v));
    return v;
  };
  const uint64_t pa = held(g.a_codes), pb = held(g.b_codes), pu = GLU ? held(f.u_codes) : pb;
  const uint64_t qa = held(g.a_scales), qb = held(g.b_scales), qu = GLU ? held(f.u_scales) : qb;
  // Base of a wave's code loads: one, or two in turn where its loads alternate
  // between G and U; a base for each load where a wave serves both sides.
  constexpr int NCB = !T::WHOLE ? CODE_LOADS : GLU ? 2 : 1;
  auto cb = [](int i) { return NCB == CODE_LOADS ? i : NCB == 2 ? (i >> 1) & 1 : 0; };
  const uint8_t *cbase[NCB], *sbase[SCALE_LOADS];
  auto bases = [&](int64_t dc, int64_t ds) __attribute__((always_inline)) {   // dc, ds: the weights' distance from the first expert's
#pragma unroll
    for (int i = 0; i < NCB; ++i) {
      const int q = NCB == 2 ? 2 * i : code_group(i);   // (a wave's load count is a multiple of 4)
      cbase[i] = reinterpret_cast<const uint8_t*>(!code_w(i) ? +pa : (q & 2) ? pu + dc : pb + dc);
    }
#pragma unroll
    for (int i = 0; i < SCALE_LOADS; ++i)
      sbase[i] = reinterpret_cast<const uint8_t*>(!scale_w(i) ? +qa : lane >= 32 ? qu + ds : qb + ds);
  };
  if constexpr (!MOE) bases(0, 0);
  // The j-th tile of this workgroup: its first activation row, the end of its
  // rows, its place along N and (MOE) its expert.
  struct Place { int row0, end, tn, expert; };
  auto place = [&](int j) __attribute__((always_inline)) {
    Place p;
    int tm;
    if constexpr (MOE) {
      const int L = j * grid + slot, rt = __builtin_amdgcn_readfirstlane(L / tiles_n);
      const moe::i32x4 e = moe::uniform4(f.tiles[HI] + 4 * (int64_t)rt);
      tile_coords(L - e[3] * tiles_n, (e[2] - e[1] + BM - 1) / BM, tiles_n, tm, p.tn);
      p.row0 = __builtin_amdgcn_readfirstlane(e[1] + tm * BM);
      p.tn = __builtin_amdgcn_readfirstlane(p.tn);
      p.end = e[2];
      p.expert = e[0];
    } else {
      tile_coords(j * grid + slot, tiles_m, tiles_n, tm, p.tn);
      p.row0 = tm * BM;
      p.end = g.m;
      p.expert = 0;
    }
    return p;
  };
  uint32_t coff[CODE_LOADS], soff[SCALE_LOADS];
  const bool a_tiled = MOE ? moe::a_tiled(f) : tiled;
  // MOE: the rows of A that this lane loads for a tile (activation side).
  struct Rows { Place at; int code[CODE_LOADS], scale[SCALE_LOADS]; };
  auto fetch = [&](int j, Rows& t) __attribute__((always_inline)) {
    t.at = place(j);
    if (!w_first) {
#pragma unroll
      for (int i = 0; i < CODE_LOADS; ++i)
        t.code[i] = moe::source_row(f, min(t.at.row0 + 16 * code_group(i) - BN + (lane >> 2), t.at.end - 1));
#pragma unroll
      for (int i = 0; i < SCALE_LOADS; ++i)
        t.scale[i] = moe::source_row(f, min(t.at.row0 + 64 * scale_group(i) - BN + lane, t.at.end - 1));
    }
  };
  auto offsets = [&](const Place& at, const Rows& t) __attribute__((always_inline)) {
    const int tn = at.tn;
    if constexpr (MOE) bases(at.expert * moe::code_step(f), at.expert * moe::scale_step(f));
#pragma unroll
    for (int i = 0; i < CODE_LOADS; ++i) {
      const int q = code_group(i);
      const bool w = code_w(i);
      const int row0 = w ? tn * TN + (GLU ? 32 * (q >> 2) + 16 * (q & 1) : 16 * q) : at.row0 + 16 * q - BN;
      if (MOE && !w) {
        // (a tile's rows lie in a swizzle of their own: the source's is undone)
        const uint32_t src = (uint32_t)t.code[i], chunk = (uint32_t)((lane & 3) ^ swz((16 * q - BN + (lane >> 2)) & 255));
        coff[i] = a_tiled ? (src >> 8) * nstage * (16 * 1024) + (src & 255) * 64 + 16 * (chunk ^ (uint32_t)swz((int)(src & 255)))
                          : src * kbytes + 16 * chunk;
      } else if (tiled) {
        coff[i] = (uint32_t)(row0 >> 8) * nstage * (16 * 1024) + (uint32_t)(row0 & 255) * 64 + lane * 16;
      } else {
        const int row = row0 + (lane >> 2);
        const uint32_t grow = (uint32_t)min(row, (w ? g.n : g.m) - 1);
        coff[i] = grow * kbytes + 16u * (uint32_t)((lane & 3) ^ swz(row & 255));
      }
    }
#pragma unroll
    for (int i = 0; i < SCALE_LOADS; ++i) {
      const int q = scale_group(i);
      const bool w = scale_w(i);
      const int row = MOE && !w ? t.scale[i] : w ? tn * TN + (GLU ? 32 * q + lr : 64 * q + lane) : at.row0 + 64 * q - BN + lane;
      soff[i] = (MOE && !w ? a_tiled : tiled) ? (uint32_t)(row >> 8) * nstage * 1024 + (uint32_t)(row & 255) * 4
                                              : (uint32_t)min(row, (MOE && !w ? row + 1 : w ? g.n : g.m) - 1) * kblocks;
    }
  };
  // bytes per stage (MOE: each wave loads one side, of a layout of its own)
  const bool strided = MOE && !w_first ? a_tiled : tiled;
  const uint32_t cstride = strided ? 16 * 1024 : RB, sstride = strided ? 1024 : 4;
  int ij = 0, ikt = 0, ibuf = 0;   // issue state: tile, stage within it, ring slot
  // MOE: a tile's rows are asked for two tiles ahead, in the epilogue, so that
  // nobody waits for them (and, vector loads arriving in order, for the ring's)
  // where the ring goes on to it; the ring is one tile ahead of the epilogue at
  // most if nk >= NBUF - 1.
  const bool early = MOE && nk >= NBUF - 1;
  Rows next;
  auto plan = [&](int j) __attribute__((always_inline)) {
    if constexpr (MOE) {
      if (!early || j == 0) fetch(j, next);
      offsets(next.at, next);
    } else {
      offsets(place(j), next);
    }
  };
  static_assert(!MOE || T::WHOLE, "a wave's loads are of one side");
  plan(0);
  auto issue_codes = [&](int i0, int i1) __attribute__((always_inline)) {
    uint8_t* dst = lds + ibuf * STAGE_BYTES;
    // (TAIL: the lane's block of the stage is the same one in all its loads)
    const bool in = !T::TAIL || 4 * ikt + ((lane & 3) ^ swz(lane >> 2)) < (int)kblocks;
#pragma unroll
    for (int i = i0; i < i1; ++i) {
      const uint8_t* src = cbase[cb(i)] + ikt * cstride + coff[i];
      if constexpr (T::TAIL) src = in ? src : reinterpret_cast<const uint8_t*>(&kZeroBlock);
      load_lds16(src, dst + code_group(i) * 1024);
    }
  };
  auto issue_scales = [&]() __attribute__((always_inline)) {
    uint8_t* dst = lds + ibuf * STAGE_BYTES + CODE_BYTES;
#pragma unroll
    for (int i = 0; i < SCALE_LOADS; ++i) {
      if constexpr (T::TAIL) {
#pragma unroll
        for (int b = 0; b < 4; ++b)   // (past K the last block's again: their codes are zeros)
          load_lds1(sbase[i] + min(4 * ikt + b, (int)kblocks - 1) + soff[i], dst + 4 * T::ROWS * b + 256 * scale_group(i));
      } else {
        load_lds4(sbase[i] + ikt * sstride + soff[i], dst + 256 * scale_group(i));
      }
    }
  };
  auto advance = [&]() __attribute__((always_inline)) {
    ibuf = ibuf + 1 == NBUF ? 0 : ibuf + 1;
    if (++ikt == nk) {
      ikt = 0;
      if ((++ij) * nk < total) plan(ij);
    }
  };

  const int wn = wave % WN, wm = wave / WN;
  int wrow[FN], xrow[FM];   // stage rows of this lane's fragments
#pragma unroll
  for (int q = 0; q < FN; ++q) wrow[q] = wn * (BN / WN) + 32 * q + lr;
#pragma unroll
  for (int q = 0; q < FM; ++q) xrow[q] = BN + wm * (BM / WM) + 32 * q + lr;
  auto load_scales = [&](const uint8_t* sbuf, uint32_t (&sw)[FN], uint32_t (&sx)[FM]) {
    auto two = [&](int row) -> uint32_t {   // scales of the lane's blocks of both sub-steps
      if constexpr (T::TAIL) {
        const uint8_t* p = sbuf + CODE_BYTES + 4 * row + 8 * T::ROWS * lg;
        return *reinterpret_cast<const uint32_t*>(p) | *reinterpret_cast<const uint32_t*>(p + 4 * T::ROWS) << 8;
      } else {
        return *reinterpret_cast<const uint16_t*>(sbuf + CODE_BYTES + 4 * row + 2 * lg);
      }
    };
#pragma unroll
    for (int q = 0; q < FN; ++q) sw[q] = two(wrow[q]);
#pragma unroll
    for (int q = 0; q < FM; ++q) sx[q] = two(xrow[q]);
  };
  auto load_frags = [&](const uint8_t* sbuf, int s, u32x4 (&wf)[FN], u32x4 (&xf)[FM]) {
    const int c = 2 * lg + s;
#pragma unroll
    for (int q = 0; q < FN; ++q)
      wf[q] = *reinterpret_cast<const u32x4*>(sbuf + wrow[q] * RB + 16 * (c ^ swz(wrow[q])));
#pragma unroll
    for (int q = 0; q < FM; ++q)
      xf[q] = *reinterpret_cast<const u32x4*>(sbuf + xrow[q] * RB + 16 * (c ^ swz(xrow[q])));
  };

  // Bias of this lane's weight row in each fragment of the wave (lanes 32-63
  // feed the MFMA's second K index: 0).
  float one;
  uint64_t zero = 0;
  asm volatile("v_mov_b32 %0, 1.0" : "=v"(one));
  asm volatile("" : "+v"(zero));
  const bool biased = f.bias != nullptr || (GLU && f.bias_u != nullptr);
  float bias[FN];
  auto load_bias = [&](int tn, int expert) {
#pragma unroll
    for (int a = 0; a < FN; ++a) {
      const void* src = GLU && (a & 1) ? f.bias_u : f.bias;
      const int n = tn * TN + wn * WCOLS + 32 * (GLU ? a >> 1 : a) + lr;
      bias[a] = 0.0f;
      if (src != nullptr && lg == 0 && n < g.n) bias[a] = vec_elem(src, f.vec_bf16, MOE ? (int64_t)expert * g.n + n : n);
    }
  };

  // The ring always has NBUF - 1 stages in flight (see gemm_large_kernel).
  each([&](auto p) __attribute__((always_inline)) {
    if constexpr (p > 0) advance();
    issue_codes(0, CODE_LOADS);
    issue_scales();
  }, std::make_integer_sequence<int, NBUF - 1>{});
  if constexpr (MOE) {
    if (early && nk < total) fetch(1, next);
  }
  v16f acc[FN][FM];
#pragma unroll
  for (int a = 0; a < FN; ++a)
#pragma unroll
    for (int c = 0; c < FM; ++c) acc_clear(acc[a][c], zero);

  wait_stages<NBUF - 2, LPS>();
  __builtin_amdgcn_s_barrier();
  uint32_t sw[FN], sx[FM];
  u32x4 wa[FN], xa[FM];
  load_scales(lds, sw, sx);
  load_frags(lds, 0, wa, xa);

  // 128 x 128 tiles: the residual of a tile is asked for PF stages before its
  // epilogue, one 4-byte load (into LDS that nobody reads) for every 128-byte
  // line of the wave's block, so that the epilogue's loads hit in L2 (2048 x
  // 14336 -> 4096: 74.7 -> 70.6 us).  The larger tiles lose more to the ring
  // loads waiting behind these than they gain (16384 x 3072 -> 12288: 409
  // against 425 us with it).
  constexpr bool AHEAD = PIECES && FM * FN == 4;
  constexpr int PF = 8;
  auto prefetch_res = [&](int row0, int tn) {
    constexpr int RSZ = RES == 1 ? 2 : 4, LINES = WCOLS * RSZ / 128;   // per row
    const int mw0 = row0 + wm * (BM / WM), nw0 = tn * TN + wn * WCOLS;
    const uint8_t* res = static_cast<const uint8_t*>(f.residual);
#pragma unroll
    for (int i = 0; i < BM / WM * LINES / 64; ++i) {
      const int line = 64 * i + lane;
      const int m = min(mw0 + line / LINES, g.m - 1), n = min(nw0 + line % LINES * (128 / RSZ), g.n - 4);
      load_lds4(res + ((int64_t)m * f.ld_res + n) * RSZ, lds + NBUF * STAGE_BYTES + 256 * wave);
    }
  };

  int cbuf = 0;   // ring slot of the stage being computed
  for (int j = 0; j * nk < total; ++j) {
    const Place at = place(j);
    const int tn = at.tn, end = at.end;
    const int ahead = AHEAD && f.residual != nullptr ? max(nk - PF, 0) : nk;
    if (biased) load_bias(tn, at.expert);
    // the compiler does not see the accumulators being cleared (inline asm):
    // wait states before the K loop's MFMAs read them
    mfma_wait();

    // MOE: a wave without rows in the tile (an expert's last) only keeps the ring
    // going.  (A loop of its own: a branch in the other one would hold up its MFMAs.)
    int k0 = 0;
    if constexpr (MOE) {
      if (at.row0 + wm * (BM / WM) >= end) {
        for (; k0 < nk; ++k0) {
          advance();
          wait_stages<NBUF - 3, LPS>();
          __builtin_amdgcn_s_barrier();
          __builtin_amdgcn_sched_barrier(0);
          cbuf = cbuf + 1 == NBUF ? 0 : cbuf + 1;
          issue_codes(0, CODE_LOADS);
          issue_scales();
          __builtin_amdgcn_sched_barrier(0);
        }
        load_scales(lds + cbuf * STAGE_BYTES, sw, sx);
        load_frags(lds + cbuf * STAGE_BYTES, 0, wa, xa);
      }
    }
    for (int kt = k0; kt < nk; ++kt) {
      if constexpr (AHEAD) {
        if (kt == ahead) prefetch_res(at.row0, tn);
      }
      advance();   // to stage it + NBUF - 1
      wait_stages<NBUF - 3, LPS>();
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);

      const uint8_t* sbuf = lds + cbuf * STAGE_BYTES;
      cbuf = cbuf + 1 == NBUF ? 0 : cbuf + 1;
      const uint8_t* nbuf = lds + cbuf * STAGE_BYTES;

      u32x4 wb[FN], xb[FM];
      load_frags(sbuf, 1, wb, xb);
      issue_codes(0, CODE_LOADS_B);
#pragma unroll
      for (int a = 0; a < FN; ++a)
#pragma unroll
        for (int c = 0; c < FM; ++c) acc[a][c] = mma<0>(wa[a], xa[c], acc[a][c], sw[a], sx[c]);
      sched_substep<FN * FM, NRD, CODE_LOADS_B>();

      uint32_t sw1[FN], sx1[FM];
#pragma unroll
      for (int q = 0; q < FN; ++q) sw1[q] = sw[q];
#pragma unroll
      for (int q = 0; q < FM; ++q) sx1[q] = sx[q];
      load_scales(nbuf, sw, sx);
      load_frags(nbuf, 0, wa, xa);
      issue_codes(CODE_LOADS_B, CODE_LOADS);
      issue_scales();
#pragma unroll
      for (int a = 0; a < FN; ++a)
#pragma unroll
        for (int c = 0; c < FM; ++c) acc[a][c] = mma<1>(wb[a], xb[c], acc[a][c], sw1[a], sx1[c]);
      sched_substep<FN * FM, NRD + T::NRS, LPS - CODE_LOADS_B>();
      __builtin_amdgcn_sched_barrier(0);
    }

    // ---- epilogue of this workgroup's j-th tile
    const int mw0 = at.row0 + wm * (BM / WM), nw0 = tn * TN + wn * WCOLS;   // the wave's block of Y
    const bool relu = f.act == act::RELU;
    const bool more = early && (j + 2) * nk < total;
    if constexpr (MOE) {
      if (more) fetch(j + 2, next);
    }
    // next's loads have arrived: called ahead of the epilogue's first stores
    auto settle = [&]() __attribute__((always_inline)) {
      if constexpr (MOE) {
#pragma unroll
        for (int i = 0; i < CODE_LOADS; ++i) asm volatile("" : "+v"(next.code[i]));
#pragma unroll
        for (int i = 0; i < SCALE_LOADS; ++i) asm volatile("" : "+v"(next.scale[i]));
      }
    };
    constexpr int NO = GLU ? FN / 2 : FN;   // output fragments along N

    // The bias onto the i-th output fragment, in the order in which they leave.
    auto add_bias = [&](int i) {
      const int o = i % NO, bb = i / NO;
      if constexpr (GLU) {
        acc_add_bias(acc[2 * o][bb], bias[2 * o], one);
        acc_add_bias(acc[2 * o + 1][bb], bias[2 * o + 1], one);
      } else {
        acc_add_bias(acc[o][bb], bias[o], one);
      }
    };
    if (biased) {
      mfma_wait();
      add_bias(0);
      mfma_wait();
    }
    // Values that an activation takes together: a branch for each group, so all
    // of a fragment's, but 4 beside an fp32 residual's pieces, whose kernels are
    // at the limit of their registers (with 16 at a time four of them spilled).
    constexpr int AW = RES == 2 ? 4 : 16;
    // Output fragment `o` (of FN, or FN / 2 gated ones) for activation rows
    // bb: accumulators read and cleared, act applied.  The next one's bias is
    // added first: the 16 reads, the wait and the clearing MFMA that follow are
    // the wait states until that one is read.
    auto take = [&](int o, int bb, float (&v)[16]) {
      if (biased && bb * NO + o + 1 < NO * FM) add_bias(bb * NO + o + 1);
      if constexpr (GLU) {
        float u[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] = acc_read(acc[2 * o][bb][r]);
        acc_clear(acc[2 * o][bb], zero);
#pragma unroll
        for (int r = 0; r < 16; ++r) u[r] = acc_read(acc[2 * o + 1][bb][r]);
        acc_clear(acc[2 * o + 1][bb], zero);
        activate<ACT, AW>(v, relu);
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] = v[r] * u[r];
      } else {
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] = acc_read(acc[o][bb][r]);
        acc_clear(acc[o][bb], zero);
        activate<ACT, AW>(v, relu);
      }
    };

    if constexpr (OUT == 2) {
      // MXFP4 output from the registers: lane l (row l % 32, half g = l / 32)
      // holds the runs n = 8 t + 4 g .. + 3 of the fragment's 32-block, its
      // partner l ^ 32 the others.  As gemm_large_kernel<2>'s epilogue.
#pragma unroll
      for (int bb = 0; bb < FM; ++bb) {
        const int m = mw0 + 32 * bb + lr;
        uint8_t *crow, *srow;   // the row's codes and scales at the 128-column stage of nw0 (tiled) or at nw0
        int swr = 0, blk0 = 0;
        if (g.q_tiled) {
          const uint32_t r8 = (uint32_t)m & 255u;
          const uint64_t ts = (uint64_t)((uint32_t)m >> 8) * ((uint32_t)g.n >> 7) + ((uint32_t)nw0 >> 7);
          crow = g.q_codes + ts * 16384 + r8 * 64;
          srow = g.q_scales + ts * 1024 + r8 * 4;
          swr = swz((int)r8);
          blk0 = (nw0 >> 5) & 3;
        } else {
          crow = g.q_codes + (int64_t)m * (g.n >> 1) + (nw0 >> 1);
          srow = g.q_scales + (int64_t)m * (g.n >> 5) + (nw0 >> 5);
        }
        const bool row_ok = m < end;
#pragma unroll
        for (int o = 0; o < NO; ++o) {
          float v[16];
          take(o, bb, v);
          if (o == 0 && bb == 0) settle();
          if (f.h32) hadamard_fragment(v);
          float am = 0.0f;
#pragma unroll
          for (int r = 0; r < 16; ++r) am = fmaxf(am, fabsf(v[r]));
          float other = am;
          swap_halves(am, other);   // both lanes of a row: its lower and its upper half's
          am = fmaxf(am, other);
          const uint32_t ef = __float_as_uint(am) >> 23;
          const uint32_t sb = ef > 2u ? ef - 2u : 0u;
          const float sc = __uint_as_float(sb ? sb << 23 : 0x00400000u);
          uint32_t w0 = 0, w1 = 0;   // runs t = 0, 1 and t = 2, 3: two code bytes per run
          w0 = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w0, v[0], v[1], sc, 0);
          w0 = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w0, v[2], v[3], sc, 1);
          w0 = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w0, v[4], v[5], sc, 2);
          w0 = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w0, v[6], v[7], sc, 3);
          w1 = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w1, v[8], v[9], sc, 0);
          w1 = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w1, v[10], v[11], sc, 1);
          w1 = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w1, v[12], v[13], sc, 2);
          w1 = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w1, v[14], v[15], sc, 3);
          // half 0 collects code bytes 0..7 of the block, half 1 bytes 8..15
          const auto lh = __builtin_amdgcn_permlane32_swap(w0, w1, false, false);
          const uint32_t lo = lh[0], hi = lh[1];
          const uint32_t d0 = (lo & 0xFFFFu) | (hi << 16), d1 = (lo >> 16) | (hi & 0xFFFF0000u);
          if (row_ok && nw0 + 32 * o < g.n) {
            const int chunk = g.q_tiled ? (blk0 + o) ^ swr : o;
            *reinterpret_cast<uint2*>(crow + 16 * chunk + 8 * lg) = make_uint2(d0, d1);
            if (lg == 0) srow[blk0 + o] = (uint8_t)sb;
          }
          __builtin_amdgcn_sched_barrier(0);   // one fragment at a time (register pressure)
        }
      }
    } else {
      // Dense output, staged per wave in the ring slot of the stage just
      // computed (free until the next issue, which follows the next barrier):
      // 32 rows of SB bytes per pass, 16-byte chunk c of row r at chunk
      // c ^ (r % chunks), which spreads both the writes (32 rows, one chunk)
      // and the reads (whole rows) over the banks.  SE: bytes of a staged
      // element (bf16 only where nothing is added after it).
      constexpr int SE = (OUT == 1 || OUT == 3) && RES == 0 ? 2 : 4;
      // fragments per pass: whole 256-byte rows where the ring slot holds them
      constexpr int MAXF = (STAGE_BYTES / (NW * 32) >= 256 ? 256 : 128) / (32 * SE);
      constexpr int FPP = NO < MAXF ? NO : MAXF;
      constexpr int SB = FPP * 32 * SE;
      constexpr int LPR = SB / 16, RPI = 64 / LPR;          // lanes (chunks) per row, rows per instruction
      constexpr int EPL = 16 / SE;                          // elements per lane
      constexpr int OSZ = OUT == 1 || OUT == 3 ? 2 : 4;     // bytes of an output element
      static_assert(NW * 32 * SB <= STAGE_BYTES, "staging area");
      const int lslot = cbuf == 0 ? NBUF - 1 : cbuf - 1;
      uint8_t* tb = lds + lslot * STAGE_BYTES + wave * (32 * SB);
      const int prow = lane / LPR, pcol = (lane % LPR) * EPL;   // this lane's piece of a row group
      constexpr int NQ = NO / FPP, NP = FM * NQ;                // passes along N, passes

      // RES 1 and 2: residual and output through buffer instructions from the
      // wave's first row on: rows past m are out of range (loads give 0, stores
      // are dropped), and so are columns past n (an offset of 2^31), so edge
      // tiles need no branches, which cost a wait for every load in flight
      // where they join.  Residual pieces are loaded RD - 1 passes ahead: the
      // bytes in flight bound its rate.
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      typedef uint32_t rvec __attribute__((ext_vector_type(RES == 1 ? 2 : 4)));   // 4 elements
      constexpr int RSZ = RES == 1 ? 2 : 4;
      constexpr int RD = FM * FN > 4 ? 2 : NP < 4 ? NP : 4;
      constexpr int kNonTemporal = 2;   // buffer cache policy nt
      rvec rres[RD][32 / RPI];
      const int rows = max(0, min(BM / WM, g.m - mw0));
      const int64_t first = PIECES && rows > 0 ? mw0 : 0;
      uint32_t ldr = (uint32_t)f.ld_res * RSZ, ldy = (uint32_t)g.ld_y * OSZ;   // row strides, bytes
      // (opaque here: else every row's offset is held in a register over all tiles)
      asm volatile("" : "+s"(ldr), "+s"(ldy));
      const __amdgpu_buffer_rsrc_t rr = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<uint8_t*>(static_cast<const uint8_t*>(f.residual)) + first * f.ld_res * RSZ, 0, rows * ldr, 0x00020000);
      const __amdgpu_buffer_rsrc_t yr =
          __builtin_amdgcn_make_buffer_rsrc(static_cast<uint8_t*>(g.y) + first * g.ld_y * OSZ, 0, rows * ldy, 0x00020000);
      auto column = [&](int q) { return nw0 + q * (FPP * 32) + pcol; };
      auto offset = [&](int p, int r, uint32_t ld, int size) {
        const int n = column(p % NQ);
        return (n < g.n ? (uint32_t)n * size : 0x80000000u) + (uint32_t)(32 * (p / NQ) + RPI * r + prow) * ld;
      };
      auto load_res = [&](int p) {
#pragma unroll
        for (int r = 0; r < 32 / RPI; ++r) {
          const int at = (int)offset(p, r, ldr, RSZ);
          if constexpr (RES == 1) rres[p % RD][r] = __builtin_amdgcn_raw_buffer_load_b64(rr, at, 0, kNonTemporal);
          else rres[p % RD][r] = __builtin_amdgcn_raw_buffer_load_b128(rr, at, 0, kNonTemporal);
        }
      };
      // Gate values of this lane's columns: a wave's rows lie in two groups at
      // most, the rows from `next` on in the second.
      f32x4 gate[2][NQ];
      int next = 0;
      if constexpr (PIECES) {
        if (f.residual != nullptr) {
#pragma unroll
          for (int p = 0; p < RD - 1 && p < NP; ++p) load_res(p);
        }
        if (f.gate != nullptr) {
          const uint32_t g0 = (uint32_t)min(mw0, g.m - 1) / f.group_rows, groups = (uint32_t)(g.m - 1) / f.group_rows;
          next = (int)min((g0 + 1) * (uint64_t)f.group_rows, (uint64_t)g.m);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int q = 0; q < NQ; ++q)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                gate[i][q][e] = vec_elem(f.gate, f.vec_bf16, (int64_t)min(g0 + i, groups) * f.ld_gate +
                                                                 min(column(q) + e, g.n - 1));
        }
      }
      // RES 0: whole aligned pieces, and nothing to leave out of the tile
      const bool vec = ((uintptr_t)g.y % 16) == 0 && ((g.ld_y * OSZ) % 16) == 0;
      const bool full = vec && at.row0 + BM <= end && (tn + 1) * TN <= g.n;
      __builtin_amdgcn_s_barrier();   // every wave is done reading that slot
      each([&](auto pass) __attribute__((always_inline)) {
        constexpr int p = pass;
        constexpr int bb = p / NQ, q = p % NQ, o0 = q * FPP;
        const int m0 = mw0 + 32 * bb + prow, n0 = column(q);
        if constexpr (PIECES) {
          if (f.residual != nullptr && p + RD - 1 < NP) load_res(p + RD - 1);
        }
        uint32_t zbytes = 0;
        static_assert(OUT != 3 || FPP == 4 || FPP == 2, "z scale bytes of a pass");
#pragma unroll
        for (int o = o0; o < o0 + FPP; ++o) {
          float v[16];
          take(o, bb, v);
          if constexpr (OUT == 3) {
            // 2^14 <= amax < 2^15 after scaling: no overflow, and 11 bits for every
            // value down to 2^-28 of the block's largest (the smallest normal number is
            // 2^-14; the exponent stays in 1 .. 254).  A choice, for half the bytes (8192 x
            // 8 of 64, 2048 -> 4096: 510 us a call, 663 with fp32 products): each product is
            // off by 2^-12 of itself, an eighth of the bf16 result's own rounding; where a
            // token's products cancel it counts against them, not against their sum.
            float am = 0.0f;
#pragma unroll
            for (int r = 0; r < 16; ++r) am = fmaxf(am, fabsf(v[r]));
            // (an infinity stays one at any scale: the largest finite value counts)
            if (__builtin_expect(__builtin_amdgcn_ballot_w64(am == __builtin_inff()) != 0, 0)) {
              am = 0.0f;
#pragma unroll
              for (int r = 0; r < 16; ++r) am = fabsf(v[r]) < __builtin_inff() ? fmaxf(am, fabsf(v[r])) : am;
            }
            float other = am;
            swap_halves(am, other);
            am = fmaxf(am, other);
            const uint32_t ef = min(max(__float_as_uint(am) >> 23, 15u), 254u);   // of 2^(ef - 127)
            const float sc = __uint_as_float((268u - ef) << 23);                   // 2^(14 - (ef - 127))
#pragma unroll
            for (int r = 0; r < 16; ++r) v[r] = v[r] * sc;
            // a row's bytes of the pass together where they are aligned: a store of
            // single bytes costs as much as one of whole lines
            const int m = mw0 + 32 * bb + lr, n = nw0 + 32 * o;
            uint8_t* zs = f.z_scales + (int64_t)m * (g.n >> 5) + (n >> 5);
            const bool ok = lg == 0 && m < end && n < g.n;
            if (g.n % (32 * FPP) != 0) {
              if (ok) *zs = (uint8_t)(ef - 14u);
            } else {
              zbytes = o == o0 ? ef - 14u : zbytes | (ef - 14u) << (8 * (o - o0));
              if (o == o0 + FPP - 1 && ok) {
                if constexpr (FPP == 4) *reinterpret_cast<uint32_t*>(zs - 3) = zbytes;
                else *reinterpret_cast<uint16_t*>(zs - 1) = (uint16_t)zbytes;
              }
            }
          }
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const int at = ((o - o0) * 32 + 8 * t + 4 * lg) * SE;
            uint8_t* dst = tb + lr * SB + (((at >> 4) ^ (lr & (LPR - 1))) << 4) + (at & 15);
            if constexpr (OUT == 3) {
              *reinterpret_cast<uint2*>(dst) =
                  make_uint2(pack_f16(v[4 * t], v[4 * t + 1]), pack_f16(v[4 * t + 2], v[4 * t + 3]));
            } else if constexpr (SE == 2) {
              *reinterpret_cast<uint2*>(dst) =
                  make_uint2(pack_bf16(v[4 * t], v[4 * t + 1]), pack_bf16(v[4 * t + 2], v[4 * t + 3]));
            } else {
              *reinterpret_cast<float4*>(dst) = make_float4(v[4 * t], v[4 * t + 1], v[4 * t + 2], v[4 * t + 3]);
            }
          }
        }
        if constexpr (p == 0) settle();
        // the area is private to this wave: its LDS writes land before its reads
        auto staged = [&](int r) {
          const int row = RPI * r + prow;
          return *reinterpret_cast<const u32x4*>(tb + row * SB + (((lane % LPR) ^ (row & (LPR - 1))) << 4));
        };
        if constexpr (RES == 0) {
          uint8_t* const y0 = static_cast<uint8_t*>(g.y) + ((int64_t)m0 * g.ld_y + n0) * OSZ;
          if (full) {
            // non-temporal: Y streams out without displacing the operand panels
            // the XCD's other workgroups still read from L2
#pragma unroll
            for (int r = 0; r < 32 / RPI; ++r)
              __builtin_nontemporal_store(staged(r), reinterpret_cast<u32x4*>(y0 + (int64_t)r * RPI * g.ld_y * OSZ));
          } else {
#pragma unroll 1
            for (int r = 0; r < 32 / RPI; ++r) {
              const u32x4 v = staged(r);
              uint8_t* yp = y0 + (int64_t)r * RPI * g.ld_y * OSZ;
              if (m0 + RPI * r >= end) continue;
              if (vec && n0 + EPL <= g.n) {
                *reinterpret_cast<u32x4*>(yp) = v;
              } else {
#pragma unroll
                for (int e = 0; e < EPL; ++e)
                  if (n0 + e < g.n) {
                    if constexpr (OSZ == 2) reinterpret_cast<uint16_t*>(yp)[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
                    else reinterpret_cast<uint32_t*>(yp)[e] = v[e];
                  }
              }
            }
          }
        } else if constexpr (PIECES) {
          // (whole loops under each branch: a branch per piece made every LDS read
          // wait for its latency; 16384 x 3072 -> 12288 with a gate 386 -> 350 us)
          constexpr int HR = 32 / RPI / (RES == 2 ? 2 : 1);   // fp32 residual: in halves (registers)
#pragma unroll
          for (int r0 = 0; r0 < 32 / RPI; r0 += HR) {
            f32x4 x[HR];
#pragma unroll
            for (int r = 0; r < HR; ++r) x[r] = __builtin_bit_cast(f32x4, staged(r0 + r));
            if (f.gate != nullptr) {
#pragma unroll
              for (int r = 0; r < HR; ++r) {
                const bool second = m0 + RPI * (r0 + r) >= next;
#pragma unroll
                for (int e = 0; e < 4; ++e) x[r][e] *= second ? gate[1][q][e] : gate[0][q][e];
              }
            }
            if (f.residual != nullptr) {
#pragma unroll
              for (int r = 0; r < HR; ++r) {
                const rvec rv = rres[p % RD][r0 + r];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if constexpr (RES == 1) x[r][e] += __uint_as_float(e & 1 ? rv[e >> 1] & 0xFFFF0000u : rv[e >> 1] << 16);
                  else x[r][e] += __uint_as_float(rv[e]);
                }
              }
            }
#pragma unroll
            for (int r = 0; r < HR; ++r) {
              const int at = (int)offset(p, r0 + r, ldy, OSZ);
              if constexpr (OUT == 1)
                __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_bf16(x[r][0], x[r][1]), pack_bf16(x[r][2], x[r][3])},
                                                      yr, at, 0, kNonTemporal);
              else
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x[r]), yr, at, 0, kNonTemporal);
            }
          }
        } else {   // element by element, bounds-checked (a rolled loop: little code)
#pragma unroll 1
          for (int r = 0; r < 32 / RPI; ++r) {
            const f32x4 x = __builtin_bit_cast(f32x4, staged(r));
            const int m = m0 + RPI * r;
            if (m >= g.m) continue;
            const int64_t ga = f.gate != nullptr ? (int64_t)((uint32_t)m / f.group_rows) * f.ld_gate : 0;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (n0 + e < g.n) {
                float v = x[e];
                if (f.gate != nullptr) v *= vec_elem(f.gate, f.vec_bf16, ga + n0 + e);
                if (f.residual != nullptr) v += vec_elem(f.residual, f.res_bf16, (int64_t)m * f.ld_res + n0 + e);
                const int64_t at = (int64_t)m * g.ld_y + n0 + e;
                if constexpr (OUT == 1) static_cast<uint16_t*>(g.y)[at] = (uint16_t)pack_bf16(v, 0.0f);
                else static_cast<float*>(g.y)[at] = v;
              }
          }
        }
      }, std::make_integer_sequence<int, NP>{});
    }
  }
  // no direct LDS load may still be writing when the workgroup's LDS is released
  __builtin_amdgcn_s_waitcnt(0);
}

template <class T, int ACT, int OUT, int RES, bool GLU>
hipError_t launch_tile(const FusedArgs& f, hipStream_t s) {
  constexpr int TN = GLU ? T::BN / 2 : T::BN;
  const int tiles_m = (f.g.m + T::BM - 1) / T::BM, tiles_n = (f.g.n + TN - 1) / TN;
  const int grid = large_grid(tiles_m * tiles_n, T::WGS);
  gemm_fused_large_kernel<T, ACT, OUT, RES, GLU><<<grid, T::NT, 0, s>>>(f, tiles_m, tiles_n, grid, (grid % 8) == 0);
  return hipGetLastError();
}

typedef Tile<256, 256, 4, 1> Large;
typedef Tile<128, 128, 4, 2> Mid;

template <int ACT, int OUT, int RES, bool GLU>
hipError_t launch_large(const FusedArgs& f, bool mid, hipStream_t s) {
  return mid ? launch_tile<Mid, ACT, OUT, RES, GLU>(f, s) : launch_tile<Large, ACT, OUT, RES, GLU>(f, s);
}

// What the kernels with RES 1 and 2 take: output and residual rows in whole
// aligned pieces of 4 columns, byte offsets within a wave's rows below 2^31, and
// gate groups of at least a wave's rows.
inline bool whole_pieces(const FusedArgs& f, bool mid) {
  auto ok = [&](const void* p, int64_t ld, int size) {
    return (uintptr_t)p % (4 * size) == 0 && ld % 4 == 0 && ld * size * 128 < (int64_t(1) << 31);
  };
  const uint32_t wave_rows = (mid ? Mid::BM : Large::BM) / 2;
  return f.g.n % 4 == 0 && ok(f.g.y, f.g.ld_y, f.g.y_bf16 ? 2 : 4) &&
         (f.residual == nullptr || ok(f.residual, f.ld_res, f.res_bf16 ? 2 : 4)) &&
         (f.gate == nullptr || f.group_rows >= wave_rows || f.group_rows >= (uint32_t)f.g.m);
}

// RES: a gate or a residual
template <int ACT, bool GLU, bool RES>
hipError_t launch_large_out(const FusedArgs& f, bool mid, hipStream_t s) {
  if constexpr (RES) {
    if (!whole_pieces(f, mid))
      return f.g.y_bf16 ? launch_large<ACT, 1, 3, GLU>(f, mid, s) : launch_large<ACT, 0, 3, GLU>(f, mid, s);
    if (f.residual == nullptr || f.res_bf16) return f.g.y_bf16 ? launch_large<ACT, 1, 1, GLU>(f, mid, s) : launch_large<ACT, 0, 1, GLU>(f, mid, s);
    return f.g.y_bf16 ? launch_large<ACT, 1, 2, GLU>(f, mid, s) : launch_large<ACT, 0, 2, GLU>(f, mid, s);
  } else {
    if (f.g.q_out) return launch_large<ACT, 2, 0, GLU>(f, mid, s);
    return f.g.y_bf16 ? launch_large<ACT, 1, 0, GLU>(f, mid, s) : launch_large<ACT, 0, 0, GLU>(f, mid, s);
  }
}

template <bool GLU, bool RES>
hipError_t launch_large_act(const FusedArgs& f, bool mid, hipStream_t s) {
  switch (f.act) {
    case act::SILU: return launch_large_out<act::SILU, GLU, RES>(f, mid, s);
    case act::GELU: return launch_large_out<act::GELU, GLU, RES>(f, mid, s);
    case act::GELU_TANH: return launch_large_out<act::GELU_TANH, GLU, RES>(f, mid, s);
    default: return launch_large_out<A_LINEAR, GLU, RES>(f, mid, s);
  }
}

}  // namespace large
}  // namespace mxfp4
