// Large-tile MXFP4 GEMMs with a feed-forward epilogue, and their gated form:
//   Y = residual + gate[g] * act(A B^T + bias)
//   H = act(A G^T + bias) * (A U^T + bias_u)
// dense, or requantized to MXFP4 along N after an optional Hadamard-32.
//
// The main loop is gemm_large.hip's (its header describes it): persistent
// 4-wave workgroups on 256 x 256 tiles, a 4-stage LDS ring of direct loads that
// runs across tile boundaries, 128 x 128 accumulators per wave.  What differs:
//  * Bias.  The accumulators of a tile start from the bias instead of zero, on
//    the matrix pipe: one v_mfma_f32_32x32x2_f32 per fragment, bias values of
//    the fragment's 32 weight rows (K index 0) against ones, writes bias[row]
//    into all 16 registers (exact: one product and zeros).  It takes the place
//    of the MFMA that clears a fragment, so a bias costs four dword loads per
//    wave and tile.
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
#pragma once
#include "gemm_large_core.h"
#include "activation.h"

#include <utility>

namespace mxfp4 {
namespace large {

constexpr int WN = 2, WM = 2, NW = WN * WM, NT = 64 * NW;
constexpr int FN = BN / WN / 32, FM = BM / WM / 32;
constexpr int CODE_LOADS = CODE_BYTES / 1024 / NW;   // per wave and stage, 16 B per lane
constexpr int SCALE_LOADS = ROWS * 4 / 256 / NW;     // per wave and stage, 4 B per lane
constexpr int LPS = CODE_LOADS + SCALE_LOADS;
constexpr int CODE_LOADS_B = CODE_LOADS / 2;         // issued during sub-step 0
constexpr int NRD = FN + FM;                         // fragment reads per sub-step

// Activation classes of the kernels that apply it in registers.
constexpr int A_LINEAR = 0;   // none or relu, by f.act
template <int ACT>
__device__ __forceinline__ void activate(float (&v)[16], bool relu) {
  if constexpr (ACT == A_LINEAR) {
    if (relu) {
#pragma unroll
      for (int r = 0; r < 16; ++r) v[r] = act::relu(v[r]);
    }
  } else {
#pragma unroll
    for (int r = 0; r < 16; ++r)
      v[r] = ACT == act::SILU ? act::silu(v[r]) : ACT == act::GELU ? act::gelu(v[r]) : act::gelu_tanh(v[r]);
  }
}

// body(0), body(1), .. as straight-line code: the unroller gives up on a loop
// this long and would index the accumulators in scratch memory.
template <typename F, int... I>
__device__ __forceinline__ void each(F&& body, std::integer_sequence<int, I...>) {
  (body(std::integral_constant<int, I>{}), ...);
}

// acc[i][j] = bias of weight row i, for every j.  The s_nop and the wait
// states at the tile start are those of acc_zero_mfma.
__device__ __forceinline__ void acc_bias_mfma(v16f& acc, float bias, float one) {
  asm volatile("s_nop 2\n\tv_mfma_f32_32x32x2_f32 %0, %1, %2, 0" : "=a"(acc) : "v"(bias), "v"(one));
}

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

// ACT: A_LINEAR or an mxfp4_act.  OUT: 0 fp32, 1 bf16, 2 MXFP4.  RES: 0 no gate
// or residual, 1 / 2 a gate and/or a residual, the residual bf16 / fp32.
template <int ACT, int OUT, int RES, bool GLU>
__global__ __launch_bounds__(NT, 1) void gemm_fused_large_kernel(FusedArgs f, int tiles_m, int tiles_n, int grid,
                                                                 int xcd_remap) {
  static_assert(RES == 0 || (OUT != 2 && !GLU), "gate and residual are for plain dense outputs");
  constexpr int TN = GLU ? BN / 2 : BN;          // output columns per tile
  constexpr int WCOLS = TN / WN;                 // and per wave
  __shared__ __attribute__((aligned(1024))) uint8_t lds[NBUF * STAGE_BYTES];

  const GemmArgs& g = f.g;
  const int ntiles = tiles_m * tiles_n;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int b = blockIdx.x;
  const int slot = xcd_remap ? (b & 7) * (grid >> 3) + (b >> 3) : b;
  if (slot >= ntiles) return;
  const int nk = g.k / KS;
  const int total = ((ntiles - slot + grid - 1) / grid) * nk;
  const uint32_t kbytes = (uint32_t)g.k / 2, kblocks = (uint32_t)g.k / 32;
  const int lr = lane & 31, lg = lane >> 5;

  // ---- direct LDS load plan, as gemm_large_kernel's.  Gated: 32-row group q
  // of the weight side holds rows of G (q even) or U (q odd); a code load
  // takes 16 rows of one group, a scale load 64 rows (lanes 0-31 G, 32-63 U).
  const bool w_side = wave < NW / 2;
  const uint8_t* cbase[2] = {w_side ? g.b_codes : g.a_codes, GLU && w_side ? f.u_codes : w_side ? g.b_codes : g.a_codes};
  const uint8_t* sbase = !w_side ? g.a_scales : GLU && lane >= 32 ? f.u_scales : g.b_scales;
  const int lim = (w_side ? g.n : g.m) - 1;
  const int part = wave % (NW / 2);
  uint32_t coff[CODE_LOADS], soff[SCALE_LOADS];
  const bool tiled = g.tiled;
  const uint32_t nstage = (uint32_t)nk;
  auto plan = [&](int j) {   // j-th tile of this workgroup
    int tm, tn;
    tile_coords(j * grid + slot, tiles_m, tiles_n, tm, tn);
    // first row, and the row of 16-row group rgp / of scale row r within it
    const int r0 = w_side ? tn * TN : tm * BM;
    auto group_row = [&](int rgp) { return GLU && w_side ? 32 * (rgp >> 2) + 16 * (rgp & 1) : 16 * rgp; };
#pragma unroll
    for (int i = 0; i < CODE_LOADS; ++i) {
      const int row0 = r0 + group_row(CODE_LOADS * part + i);
      if (tiled) {
        coff[i] = (uint32_t)(row0 >> 8) * nstage * (16 * 1024) + (uint32_t)(row0 & 255) * 64 + lane * 16;
      } else {
        const int row = row0 + (lane >> 2);
        const uint32_t grow = (uint32_t)min(row, lim);
        coff[i] = grow * kbytes + 16u * (uint32_t)((lane & 3) ^ swz(row & 255));
      }
    }
#pragma unroll
    for (int i = 0; i < SCALE_LOADS; ++i) {
      const int sr = 64 * (SCALE_LOADS * part + i);
      const int row = r0 + (GLU && w_side ? sr / 2 + lr : sr + lane);
      soff[i] = tiled ? (uint32_t)(row >> 8) * nstage * 1024 + (uint32_t)(row & 255) * 4
                      : (uint32_t)min(row, lim) * kblocks;
    }
  };
  const uint32_t cstride = tiled ? 16 * 1024 : RB, sstride = tiled ? 1024 : 4;   // bytes per stage
  int ij = 0, ikt = 0, ibuf = 0;   // issue state: tile, stage within it, ring slot
  plan(0);
  auto issue_codes = [&](int i0, int i1) {
    uint8_t* dst = lds + ibuf * STAGE_BYTES;
#pragma unroll
    for (int i = i0; i < i1; ++i)
      __builtin_amdgcn_global_load_lds(cbase[GLU ? (i >> 1) & 1 : 0] + ikt * cstride + coff[i],
                                       dst + (CODE_LOADS * wave + i) * 1024, 16, 0, 0);
  };
  auto issue_scales = [&]() {
    uint8_t* dst = lds + ibuf * STAGE_BYTES;
#pragma unroll
    for (int i = 0; i < SCALE_LOADS; ++i)
      __builtin_amdgcn_global_load_lds(sbase + ikt * sstride + soff[i],
                                       dst + CODE_BYTES + (64 * (SCALE_LOADS * wave + i)) * 4, 4, 0, 0);
  };
  auto advance = [&]() {
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
#pragma unroll
    for (int q = 0; q < FN; ++q)
      sw[q] = *reinterpret_cast<const uint16_t*>(sbuf + CODE_BYTES + 4 * wrow[q] + 2 * lg);
#pragma unroll
    for (int q = 0; q < FM; ++q)
      sx[q] = *reinterpret_cast<const uint16_t*>(sbuf + CODE_BYTES + 4 * xrow[q] + 2 * lg);
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

  // Bias of this lane's weight row in each fragment of the wave, for this
  // workgroup's j-th tile (lanes 32-63 feed the MFMA's second K index: 0).
  float one;
  asm volatile("v_mov_b32 %0, 1.0" : "=v"(one));
  float bias[FN];
  auto load_bias = [&](int j) {
    int tm, tn;
    tile_coords(j * grid + slot, tiles_m, tiles_n, tm, tn);
#pragma unroll
    for (int a = 0; a < FN; ++a) {
      const void* src = GLU && (a & 1) ? f.bias_u : f.bias;
      const int n = tn * TN + wn * WCOLS + 32 * (GLU ? a >> 1 : a) + lr;
      bias[a] = 0.0f;
      if (src != nullptr && lg == 0 && n < g.n) bias[a] = vec_elem(src, f.vec_bf16, n);
    }
  };

  // The ring always has NBUF - 1 stages in flight (see gemm_large_kernel).
#pragma unroll
  for (int p = 0; p < NBUF - 1; ++p) {
    if (p > 0) advance();
    issue_codes(0, CODE_LOADS);
    issue_scales();
  }
  v16f acc[FN][FM];
  load_bias(0);
#pragma unroll
  for (int a = 0; a < FN; ++a)
#pragma unroll
    for (int c = 0; c < FM; ++c) acc_bias_mfma(acc[a][c], bias[a], one);

  wait_stages<NBUF - 2, LPS>();
  __builtin_amdgcn_s_barrier();
  uint32_t sw[FN], sx[FM];
  u32x4 wa[FN], xa[FM];
  load_scales(lds, sw, sx);
  load_frags(lds, 0, wa, xa);

  int cbuf = 0;   // ring slot of the stage being computed
  for (int j = 0; j * nk < total; ++j) {
    // the compiler does not see the accumulators' start values being written
    // (inline asm): wait states before the K loop's MFMAs read them
    asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");

    for (int kt = 0; kt < nk; ++kt) {
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
      sched_substep<FN * FM, 2 * NRD, LPS - CODE_LOADS_B>();
      __builtin_amdgcn_sched_barrier(0);
    }

    // ---- epilogue of this workgroup's j-th tile
    int tm, tn;
    tile_coords(j * grid + slot, tiles_m, tiles_n, tm, tn);
    const int mw0 = tm * BM + wm * (BM / WM), nw0 = tn * TN + wn * WCOLS;   // the wave's block of Y
    if ((j + 1) * nk < total) load_bias(j + 1);   // the next tile's start values
    const bool relu = f.act == act::RELU;

    // Output fragment `o` (of FN, or FN / 2 gated ones) for activation rows
    // bb: accumulators read, their next start values written, act applied.
    auto take = [&](int o, int bb, float (&v)[16]) {
      if constexpr (GLU) {
        float u[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] = acc_read(acc[2 * o][bb][r]);
        acc_bias_mfma(acc[2 * o][bb], bias[2 * o], one);
#pragma unroll
        for (int r = 0; r < 16; ++r) u[r] = acc_read(acc[2 * o + 1][bb][r]);
        acc_bias_mfma(acc[2 * o + 1][bb], bias[2 * o + 1], one);
        activate<ACT>(v, relu);
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] = v[r] * u[r];
      } else {
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] = acc_read(acc[o][bb][r]);
        acc_bias_mfma(acc[o][bb], bias[o], one);
        activate<ACT>(v, relu);
      }
    };
    constexpr int NO = GLU ? FN / 2 : FN;   // output fragments along N

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
        const bool row_ok = m < g.m;
#pragma unroll
        for (int o = 0; o < NO; ++o) {
          float v[16];
          take(o, bb, v);
          if (f.h32) hadamard_fragment(v);
          float am = 0.0f;
#pragma unroll
          for (int r = 0; r < 16; ++r) am = fmaxf(am, fabsf(v[r]));
          am = fmaxf(am, __shfl_xor(am, 32));
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
          const uint32_t recv = (uint32_t)__shfl_xor((int)(lg ? w0 : w1), 32);
          const uint32_t lo = lg ? recv : w0, hi = lg ? w1 : recv;
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
      // 32 rows of SB bytes per pass, padded to PITCH.  SE: bytes of a staged
      // element (bf16 only where nothing is added after it).
      constexpr int SE = OUT == 1 && RES == 0 ? 2 : 4;
      constexpr int FPP = SE == 2 ? NO : 2;                 // fragments per pass
      constexpr int SB = FPP * 32 * SE, PITCH = SB + 16;
      constexpr int LPR = SB / 16, RPI = 64 / LPR;          // lanes per row, rows per instruction
      constexpr int EPL = 16 / SE;                          // elements per lane
      constexpr int OSZ = OUT == 1 ? 2 : 4;                 // bytes of an output element
      static_assert(NW * 32 * PITCH <= STAGE_BYTES, "staging area");
      const bool y_st = ((uintptr_t)g.y % 16) == 0 && ((g.ld_y * OSZ) % 16) == 0;
      bool full = y_st && (tm + 1) * BM <= g.m && (tn + 1) * TN <= g.n;
      constexpr int RSZ = RES == 1 ? 2 : 4;
      if constexpr (RES != 0) {
        if (f.residual != nullptr)
          full = full && ((uintptr_t)f.residual % (4 * RSZ)) == 0 && (f.ld_res % 4) == 0;
      }
      const int lslot = cbuf == 0 ? NBUF - 1 : cbuf - 1;
      uint8_t* tb = lds + lslot * STAGE_BYTES + wave * (32 * PITCH);
      const int prow = lane / LPR, pcol = (lane % LPR) * EPL;   // this lane's piece of a row group

      // residual pieces of one pass (full tiles), loaded a pass ahead
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      typedef uint32_t rvec __attribute__((ext_vector_type(RES == 1 ? 2 : 4)));   // 4 elements
      rvec rres[2][32 / RPI];
      auto load_res = [&](int p, rvec (&dst)[32 / RPI]) {
        const int m0 = mw0 + 32 * (p / (NO / FPP)), n0 = nw0 + (p % (NO / FPP)) * (FPP * 32) + pcol;
#pragma unroll
        for (int r = 0; r < 32 / RPI; ++r)
          dst[r] = __builtin_nontemporal_load(reinterpret_cast<const rvec*>(
              static_cast<const uint8_t*>(f.residual) + ((int64_t)(m0 + RPI * r + prow) * f.ld_res + n0) * RSZ));
      };
      constexpr int NP = FM * (NO / FPP);
      const bool res_ahead = RES != 0 && full && f.residual != nullptr;
      // one gate row for the wave's whole block of rows (full tiles): its values
      // for this lane's columns of each pass along N
      f32x4 grow[NO / FPP];
      bool one_group = true;
      if constexpr (RES != 0) {
        if (res_ahead) load_res(0, rres[0]);
        if (f.gate != nullptr) {
          const uint32_t g0 = (uint32_t)mw0 / f.group_rows;
          one_group = (uint32_t)min(mw0 + BM / WM, g.m) <= (g0 + 1) * (uint64_t)f.group_rows;
          if (one_group && full) {
#pragma unroll
            for (int q = 0; q < NO / FPP; ++q)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                grow[q][e] = vec_elem(f.gate, f.vec_bf16, (int64_t)g0 * f.ld_gate + nw0 + q * (FPP * 32) + pcol + e);
          }
        }
      }
      __builtin_amdgcn_s_barrier();   // every wave is done reading that slot
      each([&](auto pass) __attribute__((always_inline)) {
        constexpr int p = pass;
        constexpr int bb = p / (NO / FPP), q = p % (NO / FPP), o0 = q * FPP;
        if constexpr (RES != 0) {
          if (res_ahead && p + 1 < NP) load_res(p + 1, rres[(p + 1) & 1]);
        }
#pragma unroll
        for (int o = o0; o < o0 + FPP; ++o) {
          float v[16];
          take(o, bb, v);
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            uint8_t* dst = tb + lr * PITCH + ((o - o0) * 32 + 8 * t + 4 * lg) * SE;
            if constexpr (SE == 2) {
              *reinterpret_cast<uint2*>(dst) =
                  make_uint2(pack_bf16(v[4 * t], v[4 * t + 1]), pack_bf16(v[4 * t + 2], v[4 * t + 3]));
            } else {
              *reinterpret_cast<float4*>(dst) = make_float4(v[4 * t], v[4 * t + 1], v[4 * t + 2], v[4 * t + 3]);
            }
          }
        }
        // the area is private to this wave: its LDS writes land before its reads
        const int m0 = mw0 + 32 * bb, n0 = nw0 + 32 * o0 + pcol;
        auto staged = [&](int r) {
          return *reinterpret_cast<const u32x4*>(tb + (RPI * r + prow) * PITCH + (lane % LPR) * 16);
        };
        auto out = [&](int m) { return static_cast<uint8_t*>(g.y) + ((int64_t)m * g.ld_y + n0) * OSZ; };
        // gate of row m where the wave's rows span several groups
        auto gate_rows = [&](int m, f32x4& x) {
          const int64_t at = (int64_t)((uint32_t)m / f.group_rows) * f.ld_gate + n0;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n0 + e < g.n) x[e] *= vec_elem(f.gate, f.vec_bf16, at + e);
        };
        if (full) {
#pragma unroll
          for (int r = 0; r < 32 / RPI; ++r) {
            const int m = m0 + RPI * r + prow;
            const u32x4 s = staged(r);
            // non-temporal stores: Y streams out without displacing the operand
            // panels the XCD's other workgroups still read from L2
            if constexpr (RES == 0) {
              __builtin_nontemporal_store(s, reinterpret_cast<u32x4*>(out(m)));
            } else {
              f32x4 x = __builtin_bit_cast(f32x4, s);
              if (f.gate != nullptr) {
                if (one_group) x *= grow[q];
                else gate_rows(m, x);
              }
              if (f.residual != nullptr) {
                const rvec rv = rres[p & 1][r];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if constexpr (RES == 1)
                    x[e] += __uint_as_float(e & 1 ? rv[e >> 1] & 0xFFFF0000u : rv[e >> 1] << 16);
                  else
                    x[e] += __uint_as_float(rv[e]);
                }
              }
              if constexpr (OUT == 1)
                __builtin_nontemporal_store(u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])},
                                            reinterpret_cast<u32x2*>(out(m)));
              else
                __builtin_nontemporal_store(x, reinterpret_cast<f32x4*>(out(m)));
            }
          }
        } else {
          // edge tiles and unaligned rows: bounds-checked, element by element
          // where a 16-byte piece does not fit (a rolled loop: little code)
#pragma unroll 1
          for (int r = 0; r < 32 / RPI; ++r) {
            const int m = m0 + RPI * r + prow;
            if (m >= g.m) continue;
            const u32x4 s = staged(r);
            uint8_t* yp = out(m);
            if constexpr (RES == 0) {
              if (y_st && n0 + EPL <= g.n) {
                *reinterpret_cast<u32x4*>(yp) = s;
              } else {
#pragma unroll
                for (int e = 0; e < EPL; ++e)
                  if (n0 + e < g.n) {
                    if constexpr (SE == 2)
                      reinterpret_cast<uint16_t*>(yp)[e] = (uint16_t)(s[e >> 1] >> (16 * (e & 1)));
                    else
                      reinterpret_cast<uint32_t*>(yp)[e] = s[e];
                  }
              }
            } else {
              f32x4 x = __builtin_bit_cast(f32x4, s);
              if (f.gate != nullptr) gate_rows(m, x);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (n0 + e < g.n) {
                  if (f.residual != nullptr) x[e] += vec_elem(f.residual, RES == 1, (int64_t)m * f.ld_res + n0 + e);
                  if constexpr (OUT == 1) reinterpret_cast<uint16_t*>(yp)[e] = (uint16_t)pack_bf16(x[e], 0.0f);
                  else reinterpret_cast<float*>(yp)[e] = x[e];
                }
            }
          }
        }
      }, std::make_integer_sequence<int, NP>{});
    }
  }
  // no direct LDS load may still be writing when the workgroup's LDS is released
  __builtin_amdgcn_s_waitcnt(0);
}

template <int ACT, int OUT, int RES, bool GLU>
hipError_t launch_large(const FusedArgs& f, hipStream_t s) {
  constexpr int TN = GLU ? BN / 2 : BN;
  const int tiles_m = (f.g.m + BM - 1) / BM, tiles_n = (f.g.n + TN - 1) / TN;
  const int grid = large_grid(tiles_m * tiles_n);
  gemm_fused_large_kernel<ACT, OUT, RES, GLU><<<grid, NT, 0, s>>>(f, tiles_m, tiles_n, grid, (grid % 8) == 0);
  return hipGetLastError();
}

// RES: a gate or a residual
template <int ACT, bool GLU, bool RES>
hipError_t launch_large_out(const FusedArgs& f, hipStream_t s) {
  if constexpr (RES) {
    if (f.res_bf16) return f.g.y_bf16 ? launch_large<ACT, 1, 1, GLU>(f, s) : launch_large<ACT, 0, 1, GLU>(f, s);
    return f.g.y_bf16 ? launch_large<ACT, 1, 2, GLU>(f, s) : launch_large<ACT, 0, 2, GLU>(f, s);
  } else {
    if (f.g.q_out) return launch_large<ACT, 2, 0, GLU>(f, s);
    return f.g.y_bf16 ? launch_large<ACT, 1, 0, GLU>(f, s) : launch_large<ACT, 0, 0, GLU>(f, s);
  }
}

template <bool GLU, bool RES>
hipError_t launch_large_act(const FusedArgs& f, hipStream_t s) {
  switch (f.act) {
    case act::SILU: return launch_large_out<act::SILU, GLU, RES>(f, s);
    case act::GELU: return launch_large_out<act::GELU, GLU, RES>(f, s);
    case act::GELU_TANH: return launch_large_out<act::GELU_TANH, GLU, RES>(f, s);
    default: return launch_large_out<A_LINEAR, GLU, RES>(f, s);
  }
}

}  // namespace large
}  // namespace mxfp4
