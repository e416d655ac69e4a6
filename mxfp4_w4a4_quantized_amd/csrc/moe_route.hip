// Mixture-of-experts routing for gfx950: the choice of experts for each token,
// and the plan that puts the (token, choice) pairs in expert order.
#include "internal.h"
#include "moe_plan.h"

namespace mxfp4 {
namespace {

constexpr double kNone = -__builtin_inf();   // key of an expert that cannot be chosen

// ---------------------------------------------------------------------------
// Router.  Token t's scores s = softmax(l) or sigmoid(l); its choices are the
// topk experts with the largest key, ties to the lowest index; its weights are
// their scores, divided by their sum if asked, times a scale.
//
// Keys.  Without a bias the logits themselves: the scores' order before any
// rounding.  With a bias s + bias in 64 bits, where two experts next to each
// other on the border of the choice stay apart; so are the sums of a group's two
// best.  A 64-bit exponential per logit costs less than the launch.
//
// A wave per token, expert 64 i + lane in register i: a choice is a maximum over
// a lane's registers, then over the lanes by DPP moves; equal keys, which bf16
// logits often have, are settled by the smallest index among the lanes that hold
// the maximum.  Groups: the keys pass through LDS, lane g scans group g, and a
// group's rank among the others says whether it is kept.

// The maximum over the wave, by row shifts and row broadcasts (in lane 63).
template <int CTRL>
__device__ __forceinline__ double dpp_max(double v) {
  const uint64_t u = (uint64_t)__builtin_bit_cast(uint64_t, v);
  const int lo = (int)(uint32_t)u, hi = (int)(uint32_t)(u >> 32);
  const uint32_t l2 = (uint32_t)__builtin_amdgcn_update_dpp(lo, lo, CTRL, 0xf, 0xf, false);
  const uint32_t h2 = (uint32_t)__builtin_amdgcn_update_dpp(hi, hi, CTRL, 0xf, 0xf, false);
  return fmax(v, __builtin_bit_cast(double, ((uint64_t)h2 << 32) | l2));
}
template <int CTRL>
__device__ __forceinline__ float dpp_max(float v) {
  const int u = __float_as_int(v);
  return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(u, u, CTRL, 0xf, 0xf, false)));
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
template <typename T>
__device__ __forceinline__ T wave_max(T v) {
  v = dpp_max<0x111>(v);   // row_shr:1, 2, 4, 8
  v = dpp_max<0x112>(v);
  v = dpp_max<0x114>(v);
  v = dpp_max<0x118>(v);
  v = dpp_max<0x142>(v);   // row_bcast:15, 31
  v = dpp_max<0x143>(v);
  return lane_value(v, 63);
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

constexpr int kRouteWaves = 4;

// NV: experts per lane.  Key: float (the logits) or double (score + bias).
template <int NV, typename Key>
__global__ __launch_bounds__(64 * kRouteWaves) void moe_route_kernel(RouteArgs a) {
  extern __shared__ double lds_keys[];   // [kRouteWaves][experts], with groups
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
  if (t >= a.tokens) return;   // (no barrier below: a wave works alone)
  constexpr bool kBias = sizeof(Key) == 8;
  const float kInf = __builtin_inff();

  float x[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = 64 * i + lane;
    x[i] = -kInf;
    if (e < a.experts) {
      if (a.bf16) x[i] = __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.logits)[t * a.ld + e] << 16);
      else x[i] = static_cast<const float*>(a.logits)[t * a.ld + e];
    }
    if (!(x[i] > -kInf)) x[i] = -kInf;   // NaN is no candidate either
  }
  float bias[NV];
  if constexpr (kBias) {
#pragma unroll
    for (int i = 0; i < NV; ++i) bias[i] = 64 * i + lane < a.experts ? a.bias[64 * i + lane] : 0.0f;
  }

  // scores in 64 bits
  double s[NV];
  if (a.softmax) {
    float top = x[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) top = fmaxf(top, x[i]);
    top = wave_max(top);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      s[i] = x[i] > -kInf ? exp((double)x[i] - (double)top) : 0.0;
      sum += s[i];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] = s[i] / sum;
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] = x[i] > -kInf ? 1.0 / (1.0 + exp(-(double)x[i])) : 0.0;
  }

  Key key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if constexpr (kBias) {
      const double c = s[i] + (double)bias[i];
      key[i] = x[i] > -kInf && c > kNone ? c : kNone;
    } else {
      key[i] = x[i];
    }
  }

  if (a.groups > 1) {
    double* mine = lds_keys + (int64_t)wave * a.experts;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (64 * i + lane < a.experts) mine[64 * i + lane] = key[i] > (Key)kNone ? (kBias ? (double)key[i] : s[i]) : kNone;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    const int size = a.experts / a.groups;
    double first = kNone, second = kNone;
    if (lane < a.groups) {
      int at = lane % size;   // lanes start apart: other LDS banks
      for (int i = 0; i < size; ++i) {
        const double v = mine[lane * size + at];
        second = fmax(second, fmin(first, v));
        first = fmax(first, v);
        at = at + 1 == size ? 0 : at + 1;
      }
    }
    // a group's score: its best key, or the sum of its two best (of one where it has one)
    const double score = a.group_top2 && second > kNone ? first + second : first;
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double other = lane_value(score, g);
      rank += other > score || (other == score && g < lane) ? 1 : 0;
    }
    const uint64_t kept = __builtin_amdgcn_ballot_w64(lane < a.groups && rank < a.topk_groups);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = 64 * i + lane;
      if (e < a.experts && !((kept >> (e / size)) & 1)) key[i] = (Key)kNone;
    }
  }

  // lane j keeps choice j
  int id = -1;
  double chosen = 0.0;
  for (int j = 0; j < a.topk; ++j) {
    Key best = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < NV; ++i) {
      at = key[i] > best ? i : at;
      best = key[i] > best ? key[i] : best;
    }
    const Key top = wave_max(best);
    if (!(top > (Key)kNone)) break;
    uint64_t who = __builtin_amdgcn_ballot_w64(best == top);
    const int mine = 64 * at + lane;
    int e = __builtin_amdgcn_readlane(mine, __builtin_ctzll(who));
    for (who &= who - 1; who != 0; who &= who - 1) e = min(e, __builtin_amdgcn_readlane(mine, __builtin_ctzll(who)));
    double score = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (64 * i + lane == e) {
        score = s[i];
        key[i] = (Key)kNone;
      }
    score = lane_value(score, e & 63);
    if (lane == j) {
      id = e;
      chosen = score;
    }
  }
  if (a.renormalize) {
    const double sum = wave_sum(chosen);
    chosen = sum > 0.0 ? chosen / sum : sum != sum ? sum : 0.0;
  }
  if (lane < a.topk) {
    a.ids[t * a.topk + lane] = id;
    a.weights[t * a.topk + lane] = id < 0 ? 0.0f : (float)(chosen * (double)a.scale);
  }
}

template <int NV>
void launch_route_nv(const RouteArgs& a, hipStream_t s) {
  const int grid = (int)((a.tokens + kRouteWaves - 1) / kRouteWaves);
  const size_t lds = a.groups > 1 ? sizeof(double) * kRouteWaves * a.experts : 0;
  if (a.bias != nullptr) moe_route_kernel<NV, double><<<grid, 64 * kRouteWaves, lds, s>>>(a);
  else moe_route_kernel<NV, float><<<grid, 64 * kRouteWaves, lds, s>>>(a);
}

// ---------------------------------------------------------------------------
// Plan: a stable counting sort of the pairs by expert, on integers only (the
// same plan on every run).  Up to 4096 pairs one workgroup does it in one launch.
// Beyond that moe_count_kernel counts each chunk's pairs by expert, and in
// moe_place_kernel every workgroup adds up the counts of all chunks and of those
// before its own.  Within a chunk a wave takes a run of pairs, 64 at a time: the
// lanes with the same expert are found with a ballot for each bit of its number,
// and a lane's place among them is a bit count.

constexpr int kPlanWaves = 8;

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
  for (int64_t p = begin + threadIdx.x; p < end; p += blockDim.x) {
    const int e = expert_of(a, p, end);
    if (e >= 0) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += blockDim.x) a.counts[blockIdx.x * (int64_t)a.experts + e] = cnt[e];
}

__device__ __forceinline__ int wave_scan(int v, int lane) {   // inclusive
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

__global__ __launch_bounds__(64 * kPlanWaves) void moe_place_kernel(PlanArgs a) {
  __shared__ int32_t pos[kPlanWaves][moe::kMaxExperts];     // counts, then next rows, of each wave's run
  __shared__ int32_t total[moe::kMaxExperts], before[moe::kMaxExperts];
  __shared__ int32_t offset[moe::kMaxExperts + 1];
  __shared__ int32_t first[moe::kHeights][moe::kMaxExperts + 1];   // tiles of each height before an expert's
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int E = a.experts;
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    total[e] = before[e] = 0;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) pos[w][e] = 0;
  }
  __syncthreads();
  const int64_t run = a.chunk / kPlanWaves;   // a multiple of 64
  const int64_t begin = blockIdx.x * a.chunk + wave * run, end = min(a.pairs, begin + run);
  for (int64_t p = begin + lane; p < end; p += 64) {
    const int e = expert_of(a, p, end);
    if (e >= 0) atomicAdd(&pos[wave][e], 1);
  }
  if (gridDim.x > 1) {
    // threads over (chunk, expert) with the experts contiguous
    const int64_t n = (int64_t)gridDim.x * E;
    for (int64_t i = threadIdx.x; i < n; i += blockDim.x) {
      const int c = a.counts[i];
      const int g = (int)(i / E), e = (int)(i - (int64_t)g * E);
      if (c != 0) {
        atomicAdd(&total[e], c);
        if (g < (int)blockIdx.x) atomicAdd(&before[e], c);
      }
    }
  }
  __syncthreads();
  if (gridDim.x == 1) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
      int c = 0;
#pragma unroll
      for (int w = 0; w < kPlanWaves; ++w) c += pos[w][e];
      total[e] = c;
    }
    __syncthreads();
  }
  // wave 0: rows; wave 1 + h: tiles of height h
  if (wave <= moe::kHeights) {
    int32_t* out = wave == 0 ? offset : first[wave - 1];
    const int shift = wave == 0 ? 0 : 3 + wave;   // 16 << h rows
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + lane;
      const int c = e < E ? (total[e] + (1 << shift) - 1) >> shift : 0;
      const int v = wave_scan(c, lane);
      if (e < E) out[e] = carry + v - c;
      carry += __shfl(v, 63);
    }
    if (lane == 0) out[E] = carry;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int next = offset[e] + before[e];
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
      const int c = pos[w][e];
      pos[w][e] = next;
      next += c;
    }
  }
  __syncthreads();

  const int bits = E > 1 ? 32 - __builtin_clz(E - 1) : 0;
  const uint64_t below = (uint64_t(1) << lane) - 1;
  for (int64_t p0 = begin; p0 < end; p0 += 64) {
    const int64_t p = p0 + lane;
    const int e = expert_of(a, p, end);
    uint64_t same = __builtin_amdgcn_ballot_w64(e >= 0);
    for (int b = 0; b < bits; ++b) {
      const bool set = (e >> b) & 1;
      const uint64_t m = __builtin_amdgcn_ballot_w64(set);
      same &= set ? m : ~m;
    }
    int row = -1;
    if (e >= 0) {
      const int rank = __popcll(same & below);
      row = pos[wave][e] + rank;
      __builtin_amdgcn_wave_barrier();
      if (rank == 0) pos[wave][e] = row + __popcll(same);
      a.order[row] = (int32_t)p;
      a.token[row] = (int32_t)((uint32_t)p / (uint32_t)a.topk);
    }
    __builtin_amdgcn_wave_barrier();
    if (p < end) a.slot[p] = row;
  }

  // behind the last row, the offsets and the tile tables: shared out over the grid
  const int64_t tid = blockIdx.x * (int64_t)blockDim.x + threadIdx.x, step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t p = offset[E] + tid; p < a.pairs; p += step) {
    a.order[p] = -1;
    a.token[p] = 0;
  }
  for (int64_t e = tid; e <= E; e += step) a.offsets[e] = offset[e];
  if (tid < moe::kHeights) a.ntiles[tid] = first[tid][E];
#pragma unroll
  for (int h = 0; h < moe::kHeights; ++h) {
    const int n = first[h][E];
    for (int64_t i = tid; i < n; i += step) {
      int lo = 0, hi = E - 1;   // the last expert whose first tile is at most i, among those with tiles
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[h][mid] <= i) lo = mid;
        else hi = mid - 1;
      }
      reinterpret_cast<int4*>(a.tiles[h])[i] = make_int4(lo, offset[lo], offset[lo + 1], first[h][lo]);
    }
  }
}

// ---------------------------------------------------------------------------
// y[t] = residual[t] + sum over t's choices of weight * z[slot], z in fp32 or
// in 16 bits with a power of two per 32 columns; fp32 sums in the choices' order,
// rounded once.  A lane holds 8 columns of a row.

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
  const int32_t* slot = a.slot + t * a.topk;
  const float* weight = a.weights + t * a.topk;
#pragma unroll 4
  for (int j = 0; j < a.topk; ++j) {
    const int row = slot[j];
    const bool here = row >= 0;   // (else z's first row is read and not used)
    const float w = weight[j];
    const int64_t at = (int64_t)max(row, 0) * a.n + n0;
    if constexpr (HALF) {
      typedef _Float16 h8 __attribute__((ext_vector_type(8)));
      const h8 z = *reinterpret_cast<const h8*>(static_cast<const _Float16*>(a.z) + at);
      const float f = __uint_as_float((uint32_t)a.z_scales[at >> 5] << 23);   // (never 0: see the product's epilogue)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = here ? __builtin_fmaf(w, (float)z[i] * f, acc[i]) : acc[i];
    } else {
      const float* z = static_cast<const float*>(a.z) + at;
      if (VEC) {
        const float4 u = *reinterpret_cast<const float4*>(z), v = *reinterpret_cast<const float4*>(z + 4);
        const float zz[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = here ? __builtin_fmaf(w, zz[i], acc[i]) : acc[i];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < left && here) acc[i] = __builtin_fmaf(w, z[i], acc[i]);
      }
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
  switch ((a.experts + 63) / 64) {
    case 1: launch_route_nv<1>(a, s); break;
    case 2: launch_route_nv<2>(a, s); break;
    case 3:
    case 4: launch_route_nv<4>(a, s); break;
    case 5:
    case 6:
    case 7:
    case 8: launch_route_nv<8>(a, s); break;
    default: launch_route_nv<16>(a, s); break;
  }
  return hipGetLastError();
}

hipError_t launch_moe_plan(const PlanArgs& a, hipStream_t s) {
  const int grid = (int)moe::chunks(a.pairs);
  if (grid > 1) moe_count_kernel<<<grid, 64 * kPlanWaves, 0, s>>>(a);
  moe_place_kernel<<<grid, 64 * kPlanWaves, 0, s>>>(a);
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
