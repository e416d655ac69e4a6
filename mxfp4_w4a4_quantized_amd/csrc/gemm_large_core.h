// Shared parts of the large-tile kernels (gemm_large.hip,
// gemm_fused_large.h): tile and ring constants, the MFMA and its operand
// swizzle, accumulator access, tile order, ring waits and the schedule of a
// sub-step.  The design is described in gemm_large.hip.
#pragma once
#include "internal.h"

namespace mxfp4 {
namespace large {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int BN = 256;                      // weight rows per tile
constexpr int BM = 256;                      // activation rows per tile
constexpr int KS = 128;                      // K elements per stage
constexpr int RB = KS / 2;                   // code bytes per row per stage
constexpr int ROWS = BN + BM;                // rows per stage: W then X
constexpr int NBUF = 4;                      // LDS ring depth
constexpr int CODE_BYTES = ROWS * RB;        // 32 KiB
constexpr int STAGE_BYTES = CODE_BYTES + ROWS * 4;
constexpr int GROUP_M = 4;

static_assert(NBUF * STAGE_BYTES <= 160 * 1024, "LDS ring exceeds 160 KiB");

// Chunk swizzle: rows r and r + 4, r + 8, r + 12 (one 16-lane phase of a
// ds_read_b128 on the 64-bank LDS) and rows r, r + 2, r + 4, r + 6 (one
// 8-lane phase of a 32-bank LDS) all land in distinct 16-byte bank groups.
__device__ __forceinline__ int swz(int row) { return ((row >> 1) ^ (row >> 2)) & 3; }

template <int S>
__device__ __forceinline__ v16f mma(const u32x4& a, const u32x4& b, const v16f& c, uint32_t sa,
                                    uint32_t sb) {
  const v8i av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const v8i bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, S, (int)sa, S, (int)sb);
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Two fp32 -> packed bf16 (low half = a), round to nearest even
// (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

// One accumulator read straight from its AGPR.  The epilogues read their
// accumulators through this, one fragment at a time: with plain reads the
// register allocator copied all 256 out of the AGPRs at the loop exit in the
// MXFP4-output epilogue (which spilled), and paired each read with its pack
// through two temporaries in the bf16 one.
__device__ __forceinline__ float acc_read(float x) {
  float r;
  asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(r) : "a"(x));
  return r;
}

// Zeroed accumulators for each tile.  With a plain 0.f the compiler
// materialized the 256 zeros of a tile twice (once for a K loop that might
// not run), 512 register writes per wave and tile.  An opaque zero cannot be
// rematerialized: acc_zero() is one v_accvgpr_write (the fp32-output kernel),
// acc_zero_mfma() one MFMA of zero codes with a zero accumulator input that
// clears a whole fragment's 16 registers on the matrix pipe, which is idle
// between tiles (the bf16 and MXFP4-output kernels, whose epilogues read every
// accumulator through acc_read).  Both compiled without spills; zeros from
// the MFMA builtin, or a first K stage started from the MFMA's zero operand,
// made the compiler copy or spill the accumulators.
__device__ __forceinline__ float acc_zero() {
  float r;
  asm volatile("v_accvgpr_write_b32 %0, 0" : "=a"(r));
  return r;
}

// The compiler places no wait states before an MFMA it cannot see: the nop
// separates it from a VALU write of its operand registers just before it.
__device__ __forceinline__ void acc_zero_mfma(v16f& acc, const u32x4& zero_codes) {
  asm volatile("s_nop 2\n\tv_mfma_f32_32x32x64_f8f6f4 %0, %1, %1, 0 cbsz:4 blgp:4" : "=a"(acc) : "v"(zero_codes));
}

__device__ __forceinline__ void tile_coords(int L, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int per_group = GROUP_M * tiles_n;
  const int grp = L / per_group;
  const int first_m = grp * GROUP_M;
  const int gm = min(GROUP_M, tiles_m - first_m);
  const int r = L - grp * per_group;
  tm = first_m + r % gm;
  tn = r / gm;
}

// Wait until at most `pending` stages of this wave's direct LDS loads are
// still in flight (vector memory loads of one wave complete in order, so a
// count that only covers the later stages' loads is enough even with stores
// outstanding).
template <int PENDING, int LOADS_PER_STAGE>
__device__ __forceinline__ void wait_stages() {
  // s_waitcnt simm16 on gfx9: vmcnt[3:0] | expcnt[6:4] | lgkmcnt[11:8] | vmcnt[5:4] << 14
  constexpr int n = PENDING * LOADS_PER_STAGE;
  static_assert(n < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14));
}

// Scheduling pattern of one MFMA sub-step: MF MFMAs; RD LDS reads issued two
// per MFMA from the second MFMA on (they feed the next sub-step); VM global
// loads spread evenly over the MFMAs after the reads, so that the four waves'
// loads reach the texture unit at a steady rate.
template <int MF, int RD, int VM, int I = 0, int RDL = RD, int VML = VM>
__device__ __forceinline__ void sched_substep() {
  if constexpr (I < MF) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                   // 1 MFMA
    constexpr int rd = (I >= 1 && RDL > 0) ? (RDL >= 2 ? 2 : 1) : 0;
    if constexpr (rd > 0) __builtin_amdgcn_sched_group_barrier(0x100, rd, 0);   // LDS reads
    constexpr int from = (RD + 1) / 2 + 1;
    constexpr int span = MF - from > 0 ? MF - from : 1;
    constexpr int vm = (I >= from) ? ((I - from + 1) * VM) / span - ((I - from) * VM) / span : 0;
    constexpr int vmc = vm < VML ? vm : VML;
    if constexpr (vmc > 0) __builtin_amdgcn_sched_group_barrier(0x010, vmc, 0);  // global loads
    sched_substep<MF, RD, VM, I + 1, RDL - rd, VML - vmc>();
  } else {
    if constexpr (RDL > 0) __builtin_amdgcn_sched_group_barrier(0x100, RDL, 0);
    if constexpr (VML > 0) __builtin_amdgcn_sched_group_barrier(0x010, VML, 0);
  }
}

}  // namespace large
}  // namespace mxfp4
