// Routing of tokens to experts (sm_103a): scores, groups, the top k, weights.
//
// For each token, with s the softmax or sigmoid of its logits in fp32:
//   rank[e] = s[e] + bias[e], or without a bias the logit itself (the scores'
//             order, with nothing lost to their rounding)
//   groups: the experts are cut into `groups` runs; a run's score is the sum of
//           its two largest s + bias (s without a bias), and only the top_groups
//           best runs stay
//   ids     = the k largest ranks, ties to the lower index
//   weights = s of those, over their sum if renormalised, times scale
// An expert whose logit is -inf or NaN, or whose bias makes the rank -inf or
// NaN, is masked: it is never chosen, and a token with fewer than k experts
// left has id -1 and weight 0 in the remaining places.
//
// One warp per token; lane i holds the NV consecutive experts from NV*i (one
// vector load where the rows' alignment allows), NV the power of two that covers
// E with 32 lanes.  A lane's experts lie in one group when NV divides the group's
// size: the lane finds its two largest, and the group's lanes merge theirs by
// shuffles (a power of two of them) or through shared memory.  Ranks are compared as
// ordered integers.  Each lane puts its own in order once, in shared memory, so that
// a round of the top k is one warp-wide maximum, a vote, and a step down the list of
// the lane that wins; the lowest such lane has the lowest index.  The exponential and the division are the exact ones: a rank's last bit
// decides between experts that are nearly level.  Bound by its instructions, ~1200 a
// token of 256 experts: 16384 tokens with sigmoid, bias and groups 22.6 us (their logits
// alone would be read in 2.5 us); one token 2.5 us.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "layer.h"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kRouteThreads = 128;
constexpr uint32_t kMasked = 0;  // below every ordered rank

// Floats as unsigned integers in the same order; 0 is left for masked experts.
// (-0 ranks with +0.)
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}

__device__ __forceinline__ float load_logit(const void* p, int64_t i, int dtype) {
  if (dtype == kF32) return static_cast<const float*>(p)[i];
  if (dtype == kBF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}

// The two largest of (a1 >= b1) and (a2 >= b2).
__device__ __forceinline__ void merge_two(uint32_t& a, uint32_t& b, uint32_t a2, uint32_t b2) {
  b = max(min(a, a2), max(b, b2));
  a = max(a, a2);
}

template <int NV, int DT>
__device__ __forceinline__ void load_logits(const RouteParams& p, int64_t t, int lane, float (&x)[NV]) {
  constexpr int kSize = DT == kF32 ? 4 : 2, kBytes = NV * kSize;
  constexpr int kVec = kBytes < 16 ? kBytes : 16;  // bytes of a load
  const int e0 = lane * NV;
  if (kVec >= 4 && p.aligned % kVec == 0 && e0 + NV <= p.E) {
    const char* const src = static_cast<const char*>(p.logits) + (t * p.stride + e0) * kSize;
#pragma unroll
    for (int i = 0; i < kBytes; i += kVec) {
      uint32_t w[4];
      if constexpr (kVec == 16) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(src + i));
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
      } else if constexpr (kVec == 8) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(src + i));
        w[0] = v.x; w[1] = v.y;
      } else if constexpr (kVec == 4) {
        w[0] = __ldg(reinterpret_cast<const uint32_t*>(src + i));
      }
#pragma unroll
      for (int j = 0; j < kVec / kSize; ++j) {
        const uint32_t u = DT == kF32 ? w[j] : j % 2 ? w[j / 2] >> 16 : w[j / 2] & 0xffffu;
        x[i / kSize + j] = DT == kF32    ? __uint_as_float(u)
                           : DT == kBF16 ? __uint_as_float(u << 16)
                                         : __half2float(__ushort_as_half((unsigned short)u));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      x[i] = e0 + i < p.E ? load_logit(p.logits, t * p.stride + e0 + i, DT) : -__int_as_float(0x7f800000);
  }
}

template <int NV, int DT>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteParams p) {
  __shared__ uint32_t sorted[kRouteThreads / 32][NV][32];  // [.][rank][lane] keys
  __shared__ float scores[kRouteThreads / 32][NV][32];
  __shared__ uint8_t place[kRouteThreads / 32][NV][32];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e0 = lane * NV;
  const float inf = __int_as_float(0x7f800000);
  float bias[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) bias[i] = p.bias != nullptr && e0 + i < p.E ? p.bias[e0 + i] : 0.f;
  const int64_t step = (int64_t)gridDim.x * (kRouteThreads / 32);
  int64_t t = (int64_t)blockIdx.x * (kRouteThreads / 32) + warp;
  float next[NV];
  if (t < p.T) load_logits<NV, DT>(p, t, lane, next);
  for (; t < p.T; t += step) {
    float x[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) x[i] = next[i];
    if (t + step < p.T) load_logits<NV, DT>(p, t + step, lane, next);  // (ahead of its need)
    float top = -inf;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (x[i] != x[i]) x[i] = -inf;  // NaN: masked
      top = fmaxf(top, x[i]);
    }
    float score[NV];
    if (p.sigmoid) {
#pragma unroll
      for (int i = 0; i < NV; ++i) score[i] = 1.f / (1.f + expf(-x[i]));
    } else {
#pragma unroll
      for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        // (an infinite logit takes all; a row of -inf has no scores)
        score[i] = x[i] == top ? (top == -inf ? 0.f : 1.f) : expf(x[i] - top);
        sum += score[i];
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (sum > 0.f)
#pragma unroll
        for (int i = 0; i < NV; ++i) score[i] = score[i] / sum;
    }
    uint32_t key[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float r = x[i];
      if (p.bias != nullptr) r = x[i] == -inf ? -inf : score[i] + bias[i];
      key[i] = r == r && r != -inf ? ordered(r) : kMasked;
    }
    if (p.groups > 1) {
      const int per = p.per_group, lanes = 1 << p.lanes_log2;  // a group's experts, and lanes if whole
      const bool whole = p.lanes_log2 >= 0;
      auto group_key = [&](int i) {
        return p.bias != nullptr || key[i] == kMasked ? key[i] : ordered(score[i]);
      };
      uint32_t a = kMasked, b = kMasked;  // the two largest
      int mine;                           // the group whose key this lane has, or -1
      if (whole) {
#pragma unroll
        for (int i = 0; i < NV; ++i) merge_two(a, b, group_key(i), kMasked);
        for (int d = 1; d < lanes; d <<= 1)
          merge_two(a, b, __shfl_xor_sync(0xffffffffu, a, d), __shfl_xor_sync(0xffffffffu, b, d));
        // (lanes past the last expert are past the last group)
        mine = e0 < p.E && (lane & (lanes - 1)) == 0 ? lane >> p.lanes_log2 : -1;
      } else {
        uint32_t* const keys = &sorted[warp][0][0];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NV; ++i) keys[e0 + i] = group_key(i);
        __syncwarp();
        mine = lane < p.groups ? lane : -1;
        if (mine >= 0)
          for (int i = 0; i < per; ++i) merge_two(a, b, keys[mine * per + i], kMasked);
        __syncwarp();
      }
      uint32_t gkey = kMasked;
      if (mine >= 0 && a != kMasked)
        gkey = ordered(b != kMasked ? from_ordered(a) + from_ordered(b) : from_ordered(a));
      uint32_t open = 0;  // bit g: group g stays
      for (int j = 0; j < p.top_groups; ++j) {
        const uint32_t best = __reduce_max_sync(0xffffffffu, gkey);
        if (best == kMasked) break;
        // (the lanes that have a group's key are in the order of the groups)
        const int who = __ffs((int)__ballot_sync(0xffffffffu, gkey == best)) - 1;
        open |= 1u << (whole ? who >> p.lanes_log2 : who);
        if (lane == who) gkey = kMasked;
      }
      if (whole) {
        if (!((open >> (lane >> p.lanes_log2)) & 1u))
#pragma unroll
          for (int i = 0; i < NV; ++i) key[i] = kMasked;
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (e0 + i < p.E && !((open >> ((e0 + i) / per)) & 1u)) key[i] = kMasked;
      }
    }
    // the lane's keys in order, equal ones by index: each to its rank among them
    int rank[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) rank[i] = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = i + 1; j < NV; ++j) {
        const bool later = key[j] > key[i];
        rank[i] += later ? 1 : 0;
        rank[j] += later ? 0 : 1;
      }
    __syncwarp();  // (the last token's are read)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      sorted[warp][rank[i]][lane] = key[i];
      place[warp][rank[i]][lane] = (uint8_t)i;
      scores[warp][i][lane] = score[i];
    }
    __syncwarp();
    // the top k, best first; lane j keeps where the j-th is
    int my_lane = -1, my_head = 0, head = 0;
    uint32_t best = sorted[warp][0][lane];
    for (int j = 0; j < p.k; ++j) {
      const uint32_t all = __reduce_max_sync(0xffffffffu, best);
      if (all == kMasked) break;
      const int who = __ffs((int)__ballot_sync(0xffffffffu, best == all)) - 1;
      const int at = __shfl_sync(0xffffffffu, head, who);
      if (lane == who) {
        ++head;
        best = head < NV ? sorted[warp][head][lane] : kMasked;
      }
      if (lane == j) {
        my_lane = who;
        my_head = at;
      }
    }
    int my_at = 0;
    float w = 0.f;
    if (my_lane >= 0) {
      my_at = place[warp][my_head][my_lane];
      w = scores[warp][my_at][my_lane];
    }
    if (p.renormalize) {
      float sum = w;
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      w = sum > 0.f ? w / sum : 0.f;
    }
    if (lane < p.k) {
      p.ids[t * p.k + lane] = my_lane < 0 ? -1 : my_lane * NV + my_at;
      p.weights[t * p.k + lane] = w * p.scale;
    }
  }
}

template <int DT>
void (*route_for(int nv))(const RouteParams) {
  switch (nv) {
    case 1: return route_kernel<1, DT>;
    case 2: return route_kernel<2, DT>;
    case 4: return route_kernel<4, DT>;
    case 8: return route_kernel<8, DT>;
    case 16: return route_kernel<16, DT>;
    default: return route_kernel<32, DT>;
  }
}

}  // namespace

cudaError_t launch_route(RouteParams p, int dtype, int sms, cudaStream_t stream) {
  // the largest power of two that divides every row's address (up to 16)
  const uint64_t bits =
      (uint64_t)reinterpret_cast<uintptr_t>(p.logits) | (uint64_t)(p.stride * (dtype == kF32 ? 4 : 2)) | 16u;
  p.aligned = (int32_t)(bits & (~bits + 1));
  int nv = 1;
  while (32 * nv < p.E) nv *= 2;
  p.per_group = p.E / p.groups;
  p.lanes_log2 = -1;
  for (int i = 0; i <= 5; ++i)
    if (p.per_group == nv << i) p.lanes_log2 = i;
  auto kern = dtype == kF32 ? route_for<kF32>(nv) : dtype == kBF16 ? route_for<kBF16>(nv) : route_for<kF16>(nv);
  const int64_t warps = kRouteThreads / 32;
  int64_t ctas = (p.T + warps - 1) / warps;
  if (ctas > 8ll * sms) ctas = 8ll * sms;  // about what is resident: the bias is loaded once per warp
  return launch_pdl(kern, dim3((unsigned)ctas), dim3(kRouteThreads), 0, stream, p);
}

}  // namespace nvfp4
