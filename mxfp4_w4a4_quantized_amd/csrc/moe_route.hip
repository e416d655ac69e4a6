// Mixture-of-experts routing for gfx950: the choice of experts for each token,
// and the plan that puts the (token, choice) pairs in expert order.
#include "internal.h"
#include "moe_plan.h"
#include "moe_tile.h"

#include <type_traits>

namespace mxfp4 {
namespace {

// ---------------------------------------------------------------------------
// Router.  Token t's scores s = softmax(l) or sigmoid(l); its choices are the
// topk experts with the largest key, ties to the lowest index; its weights are
// their scores, divided by their sum if asked, times a scale.
//
// Keys are 64-bit floats: without a bias the logits themselves, the scores' order
// before any rounding; with one s + bias, where two experts next to each other on
// the border of the choice stay apart.  The expert's index is put into a key's ten
// lowest bits (which a logit leaves empty, and s + bias has at 2^-42 of its value),
// so that one maximum finds the expert and settles ties.
//
// G lanes serve a token, expert G i + lane of them in register i.  64 lanes give
// the shortest time for few tokens; for many, 16 or 32: of the instructions of a
// choice those between lanes are then shared by four or two tokens.  Bound by launch
// and load latency for few tokens (16 x 128, topk 8: 4.0 us; 2.9 of them with topk
// 1), by 64-bit arithmetic for many (8192 x 256, topk 8: softmax 9.1 us; sigmoid,
// bias and 8 groups 15.8, of them 6 the scores, 3 the groups, 4 the choice).

// Below every key: none is left.  Keys are kept within +-1e308.
constexpr uint32_t kNoneHigh = 0xFFEFFFFFu;   // of -1.79e308
__device__ __forceinline__ double none() { return __builtin_bit_cast(double, (uint64_t)kNoneHigh << 32); }
__device__ __forceinline__ bool is_none(double k) { return (uint32_t)(__builtin_bit_cast(uint64_t, k) >> 32) == kNoneHigh; }

constexpr int kIndexBits = 10;
static_assert((1 << kIndexBits) >= moe::kMaxExperts, "an expert's index fits");

__device__ __forceinline__ double pack_key(double v, int e) {
  v = v > 1e308 ? 1e308 : v < -1e308 ? -1e308 : v + 0.0;   // (+ 0.0: one zero)
  const uint64_t u = __builtin_bit_cast(uint64_t, v), mask = (1 << kIndexBits) - 1;
  const uint64_t low = (u >> 63) ? e : mask - e;            // the lower index is the larger key
  return __builtin_bit_cast(double, (u & ~mask) | low);
}
__device__ __forceinline__ int key_index(double k) {
  const uint64_t u = __builtin_bit_cast(uint64_t, k);
  const int mask = (1 << kIndexBits) - 1, low = (int)u & mask;
  return (u >> 63) ? low : mask - low;
}
__device__ __forceinline__ double key_value(double k) {
  return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, k) & ~(uint64_t)((1 << kIndexBits) - 1));
}

// The larger of two (no NaN here: a select costs less than a NaN-safe maximum).
template <typename T>
__device__ __forceinline__ T larger(T a, T b) { return a > b ? a : b; }

// v of the lane that a row rotation or a swap of rows or halves brings here.
template <int CTRL>
__device__ __forceinline__ uint32_t rotated(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ double rotated(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, ((uint64_t)rotated<CTRL>((uint32_t)(u >> 32)) << 32) | rotated<CTRL>((uint32_t)u));
}
template <int CTRL>
__device__ __forceinline__ float rotated(float v) { return __uint_as_float(rotated<CTRL>(__float_as_uint(v))); }

// v of the rows (16 lanes) or the halves of the wave, paired: of each pair both
// values in both lanes.
template <int ROWS>
__device__ __forceinline__ void paired(uint32_t v, uint32_t& a, uint32_t& b) {
  const auto r = ROWS == 1 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                           : __builtin_amdgcn_permlane32_swap(v, v, false, false);
  a = r[0];
  b = r[1];
}
template <int ROWS>
__device__ __forceinline__ void paired(float v, float& a, float& b) {
  uint32_t x, y;
  paired<ROWS>(__float_as_uint(v), x, y);
  a = __uint_as_float(x);
  b = __uint_as_float(y);
}
template <int ROWS>
__device__ __forceinline__ void paired(double v, double& a, double& b) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  uint32_t xl, yl, xh, yh;
  paired<ROWS>((uint32_t)u, xl, yl);
  paired<ROWS>((uint32_t)(u >> 32), xh, yh);
  a = __builtin_bit_cast(double, ((uint64_t)xh << 32) | xl);
  b = __builtin_bit_cast(double, ((uint64_t)yh << 32) | yl);
}

struct Max {
  template <typename T> __device__ __forceinline__ T operator()(T a, T b) const { return larger(a, b); }
};
struct Sum {
  template <typename T> __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};

// op over the G lanes of a token, in every one of them: rotations within rows of
// 16, then rows and halves of the wave swapped.
template <int G, class Op, typename T>
__device__ __forceinline__ T across(T v, Op op) {
  v = op(v, rotated<0x128>(v));   // row_ror:8, 4, 2, 1
  v = op(v, rotated<0x124>(v));
  v = op(v, rotated<0x122>(v));
  v = op(v, rotated<0x121>(v));
  T a, b;
  if constexpr (G >= 32) {
    paired<1>(v, a, b);
    v = op(a, b);
  }
  if constexpr (G == 64) {
    paired<2>(v, a, b);
    v = op(a, b);
  }
  return v;
}

// e^x in 64 bits, relative error some 2^-47: x = n ln 2 + r, |r| <= ln 2 / 2, with
// ln 2 in two parts (Cody and Waite), and the series of e^r to r^11; below 2^-1022
// in binary64's subnormal steps.  N values step by step together: one alone waits
// for each of its operations.
template <int N>
__device__ __forceinline__ void exp64(double (&x)[N]) {
  constexpr double kSeries[] = {1.0 / 39916800, 1.0 / 3628800, 1.0 / 362880, 1.0 / 40320, 1.0 / 5040, 1.0 / 720,
                                1.0 / 120,      1.0 / 24,      1.0 / 6,      0.5,         1.0,        1.0};
  double big[N], r[N], p[N];
#pragma unroll
  for (int i = 0; i < N; ++i) big[i] = __builtin_fma(x[i], 1.4426950408889634, 0x1.8p52);   // n in its lowest bits
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = __builtin_fma(big[i] - 0x1.8p52, -0.69314718036912382, x[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = __builtin_fma(big[i] - 0x1.8p52, -1.9082149292705877e-10, r[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) p[i] = kSeries[0];
#pragma unroll
  for (int t = 1; t < 12; ++t) {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = __builtin_fma(p[i], r[i], kSeries[t]);
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int i = 0; i < N; ++i)   // (far below, n's lowest bits are not n; x = -infinity)
    x[i] = x[i] < -746.0 ? 0.0 : __builtin_ldexp(p[i], (int)(uint32_t)__builtin_bit_cast(uint64_t, big[i]));
}
// 1 / (1 + e^-x).  v_rcp_f64 is right to some 2^-23, a Newton step makes that 2^-45,
// beyond what a key keeps.
template <int N>
__device__ __forceinline__ void sigmoid64(double (&x)[N]) {
  double e[N], r[N];
#pragma unroll
  for (int i = 0; i < N; ++i) e[i] = -__builtin_fabs(x[i]);
  exp64(e);
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = __builtin_amdgcn_rcp(1.0 + e[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = __builtin_fma(__builtin_fma(-(1.0 + e[i]), r[i], 1.0), r[i], r[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = x[i] < 0.0 ? e[i] * r[i] : r[i];
}

constexpr int kRouteWaves = 4;

template <int G, int NV, bool BIAS, bool GROUPS>
__global__ __launch_bounds__(64 * kRouteWaves) void moe_route_kernel(RouteArgs a) {
  extern __shared__ double lds[];   // GROUPS: [tokens][experts + groups + 1], then [tokens][64]
  constexpr int PER = 64 * kRouteWaves / G;   // tokens of a workgroup
  const int sub = threadIdx.x % G, slot = threadIdx.x / G;
  const int64_t t0 = (int64_t)blockIdx.x * PER + slot;
  const bool live = t0 < a.tokens;
  const int64_t t = live ? t0 : a.tokens - 1;   // (idle lanes repeat the last token: barriers and lane moves stay whole)
  const float kInf = __builtin_inff();

  auto logit = [&](int e) {
    const float v = a.bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.logits)[t * a.ld + e] << 16)
                           : static_cast<const float*>(a.logits)[t * a.ld + e];
    return v > -kInf ? v : -kInf;   // NaN is no candidate either
  };
  float x[NV], bias[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = G * i + sub;
    x[i] = e < a.experts ? logit(e) : -kInf;
    if constexpr (BIAS) bias[i] = e < a.experts ? a.bias[e] : 0.0f;
  }
  float top = x[0];
#pragma unroll
  for (int i = 1; i < NV; ++i) top = larger(top, x[i]);
  if (a.softmax) top = across<G>(top, Max());

  // The scores that are needed before the choice: all of them for keys with a
  // bias and for groups, and for the sum that a softmax is divided by.
  constexpr bool ALL = BIAS || GROUPS;
  double s[ALL ? NV : 1], scale = 1.0;
  if (ALL || (a.softmax && !a.renormalize)) {
    double sum = 0.0;
    constexpr int N = NV < 4 ? NV : 4;
#pragma unroll
    for (int i0 = 0; i0 < NV; i0 += N) {
      double v[N];
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = a.softmax ? (double)x[i0 + i] - (double)top : (double)x[i0 + i];
      if (a.softmax) exp64(v);
      else if constexpr (ALL) sigmoid64(v);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[i] = x[i0 + i] > -kInf ? v[i] : 0.0;
        sum += v[i];
        if constexpr (ALL) s[i0 + i] = v[i];
      }
    }
    if (a.softmax) scale = 1.0 / across<G>(sum, Sum());
  }
  double key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    double v = (double)x[i];
    if constexpr (BIAS) v = s[i] * scale + (double)bias[i];
    const bool can = x[i] > -kInf && v > -(double)kInf;
    key[i] = can ? pack_key(v, G * i + sub) : none();
  }

  if constexpr (GROUPS) {
    // Lane sub scans a part of group sub / L; a group is a run of experts, one
    // double apart from the next in LDS (other banks).
    const int size = a.experts / a.groups, stride = a.experts + a.groups + 1;
    const float per = 1.0f / (float)size;
    auto group_of = [&](int e) { return (int)(((float)e + 0.5f) * per); };
    double* mine = lds + slot * stride;
    double* scores = lds + PER * stride + slot * 64;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = G * i + sub;
      if (e < a.experts) mine[e + group_of(e)] = is_none(key[i]) ? none() : BIAS ? key_value(key[i]) : s[i];
    }
    __syncthreads();
    int L = 1;
    while (2 * L * a.groups <= G && 2 * L <= size) L *= 2;
    for (int g0 = 0; g0 < a.groups; g0 += G / L) {
      const int g = g0 + sub / L, part = sub % L;
      double first = none(), second = none();
      if (g < a.groups) {
        const double* p = mine + g * (size + 1);
        for (int i = part; i < size; i += L) {
          const double v = p[i];
          second = larger(second, first < v ? first : v);
          first = larger(first, v);
        }
      }
      for (int d = 1; d < L; d *= 2) {
        const double f2 = __shfl_xor(first, d), s2 = __shfl_xor(second, d);
        second = larger(larger(second, s2), first < f2 ? first : f2);
        first = larger(first, f2);
      }
      // its best key, or the sum of its two best (of one where it has one)
      if (part == 0 && g < a.groups) scores[g] = a.group_top2 && !is_none(second) ? first + second : first;
    }
    __syncthreads();
    uint64_t kept = 0;
    for (int g0 = 0; g0 < a.groups; g0 += G) {
      const int g = g0 + sub;
      const double score = g < a.groups ? scores[g] : none();
      int rank = 0;
      for (int h = 0; h < a.groups; ++h) {
        const double other = scores[h];
        rank += other > score || (other == score && h < g) ? 1 : 0;
      }
      const uint64_t in = __builtin_amdgcn_ballot_w64(g < a.groups && rank < a.topk_groups);
      constexpr uint64_t kToken = ~uint64_t(0) >> (64 - G);   // the token's lanes
      kept |= ((in >> (threadIdx.x & 63 & ~(G - 1))) & kToken) << g0;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (!((kept >> (group_of(G * i + sub) & 63)) & 1)) key[i] = none();   // (no expert: none already)
  }

  // lane j of the token keeps choice j
  int id = -1;
  for (int j = 0; j < a.topk; ++j) {
    double best = key[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) best = larger(best, key[i]);
    best = across<G>(best, Max());
    const int e = key_index(best), mine = e - sub;   // this lane's register e / G, if it has it
#pragma unroll
    for (int i = 0; i < NV; ++i) {   // (the upper half alone makes it none)
      const uint64_t u = __builtin_bit_cast(uint64_t, key[i]);
      const uint32_t high = mine == G * i ? kNoneHigh : (uint32_t)(u >> 32);
      key[i] = __builtin_bit_cast(double, ((uint64_t)high << 32) | (uint32_t)u);
    }
    if (sub == j) id = is_none(best) ? -1 : e;
  }
  double w = 0.0;
  if (id >= 0) {
    double l[1] = {(double)logit(id)};
    if (a.softmax) {
      l[0] -= (double)top;
      exp64(l);
      w = l[0] * scale;
    } else {
      sigmoid64(l);
      w = l[0];
    }
  }
  if (a.renormalize) {
    const double sum = across<G>(w, Sum());
    w = sum == 0.0 ? 0.0 : w / sum;
  }
  if (live && sub < a.topk) {
    a.ids[t * a.topk + sub] = id;
    a.weights[t * a.topk + sub] = (float)(w * (double)a.scale);
  }
}

template <int G, int NV>
void launch_route_nv(RouteArgs a, hipStream_t s) {
  constexpr int PER = 64 * kRouteWaves / G;
  constexpr int64_t kMost = (int64_t(1) << 23) * PER;   // tokens of a launch: a grid holds less than 2^32 threads
  const size_t bytes = sizeof(double) * PER * (a.experts + a.groups + 1 + 64);
  for (int64_t left = a.tokens; left > 0; left -= kMost) {
    a.tokens = left < kMost ? left : kMost;
    const int grid = (int)((a.tokens + PER - 1) / PER);
    if (a.groups > 1) {
      if (a.bias != nullptr) moe_route_kernel<G, NV, true, true><<<grid, 64 * kRouteWaves, bytes, s>>>(a);
      else moe_route_kernel<G, NV, false, true><<<grid, 64 * kRouteWaves, bytes, s>>>(a);
    } else {
      if (a.bias != nullptr) moe_route_kernel<G, NV, true, false><<<grid, 64 * kRouteWaves, 0, s>>>(a);
      else moe_route_kernel<G, NV, false, false><<<grid, 64 * kRouteWaves, 0, s>>>(a);
    }
    a.logits = static_cast<const uint8_t*>(a.logits) + a.tokens * a.ld * (a.bf16 ? 2 : 4);
    a.ids += a.tokens * a.topk;
    a.weights += a.tokens * a.topk;
  }
}

// ---------------------------------------------------------------------------
// Plan: a stable counting sort of the pairs by expert, on integers only (the
// same plan on every run).  Up to kOneChunk pairs one workgroup does it in one
// launch.  Beyond that moe_count_kernel counts each chunk's pairs by expert, and
// in moe_place_kernel every workgroup adds up the counts of all chunks and of
// those before its own.  Within a chunk a wave takes a run of pairs, 64 at a time:
// the lanes with the same expert are found with a ballot for each bit of its
// number, and a lane's place among them is a bit count.  Bound by latency: the
// ids, then LDS round trips between barriers.

constexpr int kPlanWaves = 16;
static_assert(64 * kPlanWaves >= moe::kMaxExperts, "a thread for each expert");
constexpr int kHeld = 4;   // steps of 64 pairs whose ids a wave reads once (8: 0.5 us slower, by its code)

__device__ __forceinline__ int expert_of(const PlanArgs& a, int64_t p, int64_t end) {
  if (p >= end) return -1;
  const uint32_t e = (uint32_t)a.ids[p] - (uint32_t)a.first;   // (ids below first wrap to far above experts)
  return e < (uint32_t)a.experts ? (int)e : -1;
}

__global__ __launch_bounds__(64 * kPlanWaves) void moe_count_kernel(PlanArgs a) {
  __shared__ int32_t cnt[moe::kMaxExperts];
  for (int e = threadIdx.x; e < a.experts; e += blockDim.x) cnt[e] = 0;
  __syncthreads();
  const int64_t begin = blockIdx.x * a.chunk, end = min(a.pairs, begin + a.chunk);
#pragma unroll 4
  for (int64_t p = begin + threadIdx.x; p < end; p += blockDim.x) {
    const int e = expert_of(a, p, end);
    if (e >= 0) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += blockDim.x) a.counts[blockIdx.x * (int64_t)a.experts + e] = cnt[e];
}

// Inclusive sum over the wave: row shifts, then row broadcasts.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);   // row_shr:1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast:31 into rows 2 and 3
  return v;
}

// What a wave's lanes wrote to LDS before it, its lanes read after it.  (The hardware
// does a wave's LDS operations in order; the fences keep the compiler from moving
// them: a wave barrier alone says nothing about memory.)
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__global__ __launch_bounds__(64 * kPlanWaves) void moe_place_kernel(PlanArgs a) {
  __shared__ int32_t pos[kPlanWaves][moe::kMaxExperts];     // counts, then next rows, of each wave's run
  __shared__ int32_t total[moe::kMaxExperts], before[moe::kMaxExperts];
  __shared__ int32_t offset[moe::kMaxExperts + 1];
  __shared__ int32_t first[moe::kHeights][moe::kMaxExperts + 1];   // tiles of each height before an expert's
  __shared__ int32_t most;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int E = a.experts;
  const bool alone = gridDim.x == 1;
  const int64_t chunk0 = blockIdx.x * a.chunk, left = a.pairs - chunk0;
  const uint32_t here = (uint32_t)(left < a.chunk ? left : a.chunk);            // pairs of this workgroup
  const uint32_t run = (here + blockDim.x - 1) / blockDim.x * 64;               // and of a wave
  const int used = run == 0 ? 0 : (int)((here + run - 1) / run);                // waves that have some
  const int64_t begin = chunk0 + wave * (int64_t)run, end = min(chunk0 + here, begin + run);
  int held[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) held[i] = expert_of(a, begin + 64 * i + lane, end);
  // a thread adds up one expert's counts over a part of the chunks, this one's
  // and the later ones' apart
  int mine = -1, sum = 0, sum_before = 0;
  if (!alone) {
    const int wide = min(E, (int)blockDim.x), parts = (int)blockDim.x / wide, grid = (int)gridDim.x;
    const int part = (int)threadIdx.x / wide;
    if (part < parts) {
      mine = (int)threadIdx.x - part * wide;
#pragma unroll 8
      for (int g = part; g < grid; g += parts) {
        const int c = a.counts[(int64_t)g * E + mine];
        sum += c;
        sum_before += g < (int)blockIdx.x ? c : 0;
      }
    }
  }
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    total[e] = before[e] = 0;
    for (int w = 0; w < used; ++w) pos[w][e] = 0;
  }
  if (threadIdx.x == 0) most = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (held[i] >= 0) atomicAdd(&pos[wave][held[i]], 1);
  for (int64_t p = begin + 64 * kHeld + lane; p < end; p += 64) {
    const int e = expert_of(a, p, end);
    if (e >= 0) atomicAdd(&pos[wave][e], 1);
  }
  if (mine >= 0) {
    atomicAdd(&total[mine], sum);
    atomicAdd(&before[mine], sum_before);
  }
  __syncthreads();
  // wave 0: rows; wave 1 + h: tiles of height h
  if (wave <= moe::kHeights) {
    int32_t* out = wave == 0 ? offset : first[wave - 1];
    const int shift = wave == 0 ? 0 : moe::shift_of(wave - 1);
    int carry = 0, top = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + lane;
      int c = 0;
      if (e < E) {
        c = total[e];
        if (alone)
          for (int w = 0; w < used; ++w) c += pos[w][e];
        c = (c + (1 << shift) - 1) >> shift;
      }
      const int v = wave_scan(c);
      if (e < E) out[e] = carry + v - c;
      carry += __builtin_amdgcn_readlane(v, 63);
      top = max(top, c);
    }
    if (lane == 0) out[E] = carry;
    if (wave == 1) atomicMax(&most, top);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int next = offset[e] + before[e];
    for (int w = 0; w < used; ++w) {
      const int c = pos[w][e];
      pos[w][e] = next;
      next += c;
    }
  }
  __syncthreads();

  const int bits = E > 1 ? 32 - __builtin_clz(E - 1) : 0;
  const uint64_t below = (uint64_t(1) << lane) - 1;
  auto place = [&](int64_t p, int e) {   // 64 pairs in their order
    uint64_t same = __builtin_amdgcn_ballot_w64(e >= 0);
    for (int b = 0; b < bits; ++b) {
      const bool set = (e >> b) & 1;
      const uint64_t m = __builtin_amdgcn_ballot_w64(set);
      same &= set ? m : ~m;
    }
    int row = -1;
    const int rank = __popcll(same & below);
    if (e >= 0) row = pos[wave][e] + rank;
    wave_lds_sync();   // every lane has read its expert's next row ..
    if (e >= 0) {
      if (rank == 0) pos[wave][e] = row + __popcll(same);
      a.order[row] = (int32_t)p;
      a.token[row] = (int32_t)((uint32_t)p / (uint32_t)a.topk);
    }
    wave_lds_sync();   // .. and the next 64 pairs read what the first of them wrote
    if (p < end) a.slot[p] = row;
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (begin + 64 * i < end) place(begin + 64 * i + lane, held[i]);
  for (int64_t p0 = begin + 64 * kHeld; p0 < end; p0 += 64) place(p0 + lane, expert_of(a, p0 + lane, end));

  // behind the last row, the offsets and the tile tables: shared out over the grid
  const int64_t tid = blockIdx.x * (int64_t)blockDim.x + threadIdx.x, step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t p = offset[E] + tid; p < a.pairs; p += step) {
    a.order[p] = -1;
    a.token[p] = 0;
  }
  for (int64_t e = tid; e <= E; e += step) a.offsets[e] = offset[e];
  if (tid < moe::kHeights) a.ntiles[tid] = first[tid][E];
  auto entry = [&](int h, int i, int e) {
    int32_t* tiles = a.tiles[0];   // (selects: an indexed kernel argument would go through memory)
#pragma unroll
    for (int j = 1; j < moe::kHeights; ++j) tiles = h == j ? a.tiles[j] : tiles;
    reinterpret_cast<int4*>(tiles)[i] = make_int4(e, offset[e], offset[e + 1], first[h][e]);
  };
  if (alone && most <= 8) {
    // few tiles each: a thread per expert and height writes them
    for (int i = threadIdx.x; i < moe::kHeights * E; i += blockDim.x) {
      const int h = i / E, e = i - h * E;
      for (int k = first[h][e]; k < first[h][e + 1]; ++k) entry(h, k, e);
    }
  } else {
    // a wave per expert and height
    const int waves = (int)blockDim.x >> 6;
    for (int i = blockIdx.x * waves + wave; i < moe::kHeights * E; i += gridDim.x * waves) {
      const int h = i / E, e = i - h * E;
      for (int k = first[h][e] + lane; k < first[h][e + 1]; k += 64) entry(h, k, e);
    }
  }
}

// ---------------------------------------------------------------------------
// y[t] = residual[t] + sum over t's choices of weight * z[slot], z in fp32 or
// in 16 bits with a power of two per 32 columns; fp32 sums in the choices' order,
// rounded once.  A lane holds 8 columns of a row.

constexpr int kAhead = 8;

template <bool HALF, bool VEC>
__global__ __launch_bounds__(256) void moe_combine_kernel(CombineArgs a) {
  const int64_t t = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
  const int n0 = (blockIdx.x * 256 + threadIdx.x) * 8;
  if (t >= a.tokens || n0 >= a.n) return;
  const int left = min(8, a.n - n0);
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
  if (a.residual != nullptr) {
    if (a.res_bf16) {
      const uint16_t* r = static_cast<const uint16_t*>(a.residual) + t * a.ld_res + n0;
      if (VEC) {
        const uint4 v = *reinterpret_cast<const uint4*>(r);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < left) acc[i] = __uint_as_float((uint32_t)r[i] << 16);
      }
    } else {
      const float* r = static_cast<const float*>(a.residual) + t * a.ld_res + n0;
      if (VEC) {
        const float4 u = *reinterpret_cast<const float4*>(r), v = *reinterpret_cast<const float4*>(r + 4);
        acc[0] = u.x, acc[1] = u.y, acc[2] = u.z, acc[3] = u.w, acc[4] = v.x, acc[5] = v.y, acc[6] = v.z, acc[7] = v.w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < left) acc[i] = r[i];
      }
    }
  }
  // Slots and weights are the same for the whole workgroup (scalar loads); kAhead
  // rows are asked for together.
  const int32_t* slot = a.slot + t * a.topk;
  const int32_t* weight = reinterpret_cast<const int32_t*>(a.weights + t * a.topk);
  typedef _Float16 h8 __attribute__((ext_vector_type(8)));
  typedef float f8 __attribute__((ext_vector_type(8)));
  typedef std::conditional_t<HALF, h8, f8> Row;
  for (int j0 = 0; j0 < a.topk; j0 += kAhead) {
    Row z[kAhead];
    uint32_t scale[kAhead];
    int row[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      row[j] = j0 + j < a.topk ? moe::uniform(slot + j0 + j) : -1;
      if (row[j] < 0) continue;
      const int64_t at = (int64_t)row[j] * a.n + n0;
      if constexpr (HALF) {
        z[j] = *reinterpret_cast<const h8*>(static_cast<const _Float16*>(a.z) + at);
        scale[j] = a.z_scales[at >> 5];
      } else {
        const float* p = static_cast<const float*>(a.z) + at;
        if (VEC) {
          const float4 u = *reinterpret_cast<const float4*>(p), v = *reinterpret_cast<const float4*>(p + 4);
          z[j] = f8{u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) z[j][i] = p[min(i, left - 1)];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (row[j] < 0) continue;
      const float w = __int_as_float(moe::uniform(weight + j0 + j));
      // (a scale byte is never 0: see the product's epilogue)
      const float f = HALF ? __uint_as_float(scale[j] << 23) : 1.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(w, HALF ? (float)z[j][i] * f : (float)z[j][i], acc[i]);
    }
  }
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  if (a.y_bf16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{acc[2 * i], acc[2 * i + 1]}, b2));
    uint16_t* y = static_cast<uint16_t*>(a.y) + t * a.ld_y + n0;
    if (VEC) {
      *reinterpret_cast<uint4*>(y) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) y[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
  } else {
    float* y = static_cast<float*>(a.y) + t * a.ld_y + n0;
    if (VEC) {
      *reinterpret_cast<float4*>(y) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      *reinterpret_cast<float4*>(y + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) y[i] = acc[i];
    }
  }
}

}  // namespace

hipError_t launch_moe_route(const RouteArgs& a, hipStream_t s) {
  const int e = a.experts;
  // Lanes a token, and us on that many and on 64 (topk 8; softmax / sigmoid with a
  // bias and 8 groups):
  //   64 experts, 16 lanes:  2048 tokens 4.3, 4.3 / 6.5, 6.2;  3000 4.3, 5.0 / 6.5, 7.0
  //   128 experts, 16 lanes: 3000 tokens 5.5, 5.6 / 8.8, 8.0;  4096 5.6, 6.4 / 8.9, 9.1;  8192 6.2, 9.7 / 10.3, 14.0
  //   256 experts, 32 lanes: 3000 tokens 6.7, 6.5 / 11.1, 9.8; 4096 6.7, 7.4 / 11.3, 11.3; 8192 8.9, 11.2 / 15.6, 17.8
  // Of more experts 32 lanes have no such crossing (512 experts, 8192 tokens: 13.3, 14.8 /
  // 28.8, 26.9); fewer lanes than 64 hold at most 16 choices here.
  if (a.tokens >= (e <= 64 ? 3000 : 4096) && e <= 256 && a.topk <= 16) {
    if (e <= 64) launch_route_nv<16, 4>(a, s);
    else if (e <= 128) launch_route_nv<16, 8>(a, s);
    else launch_route_nv<32, 8>(a, s);
  } else {
    if (e <= 64) launch_route_nv<64, 1>(a, s);
    else if (e <= 128) launch_route_nv<64, 2>(a, s);
    else if (e <= 256) launch_route_nv<64, 4>(a, s);
    else if (e <= 512) launch_route_nv<64, 8>(a, s);
    else launch_route_nv<64, 16>(a, s);
  }
  return hipGetLastError();
}

hipError_t launch_moe_plan(const PlanArgs& a, hipStream_t s) {
  const int grid = (int)moe::chunks(a.pairs);
  if (grid > 1) moe_count_kernel<<<grid, 64 * kPlanWaves, 0, s>>>(a);
  // (8 waves for few pairs: at least one each for the rows and the heights)
  moe_place_kernel<<<grid, a.pairs <= 512 ? 512 : 64 * kPlanWaves, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_moe_combine(const CombineArgs& a, hipStream_t s) {
  const int gy = (int)(a.tokens < 65535 ? a.tokens : 65535);
  const dim3 grid((a.n + 2047) / 2048, gy, (unsigned)((a.tokens + gy - 1) / gy));
  auto ok = [](const void* p, int64_t ld, int size) { return (uintptr_t)p % 16 == 0 && (ld * size) % 16 == 0; };
  const bool vec = a.n % 8 == 0 && ok(a.y, a.ld_y, a.y_bf16 ? 2 : 4) &&
                   (a.residual == nullptr || ok(a.residual, a.ld_res, a.res_bf16 ? 2 : 4));
  if (a.half) {   // (n is a multiple of 32)
    if (vec) moe_combine_kernel<true, true><<<grid, 256, 0, s>>>(a);
    else moe_combine_kernel<true, false><<<grid, 256, 0, s>>>(a);
  } else {
    if (vec) moe_combine_kernel<false, true><<<grid, 256, 0, s>>>(a);
    else moe_combine_kernel<false, false><<<grid, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace mxfp4
