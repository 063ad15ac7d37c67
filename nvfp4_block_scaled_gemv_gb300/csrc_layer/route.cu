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
// One warp per token; lane i holds the experts i, i + 32, ...  A round of the
// top k is a warp maximum over (rank, lowest index), done on the ranks as
// ordered integers with the warp-wide reduction instructions.
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

template <int NV, int DT>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteParams p) {
  __shared__ uint32_t group_keys[kRouteThreads / 32][NV * 32];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float inf = __int_as_float(0x7f800000);
  for (int64_t t = (int64_t)blockIdx.x * (kRouteThreads / 32) + warp; t < p.T;
       t += (int64_t)gridDim.x * (kRouteThreads / 32)) {
    float x[NV];
    float top = -inf;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 32 * i;
      x[i] = e < p.E ? load_logit(p.logits, t * p.stride + e, DT) : -inf;
      if (x[i] != x[i]) x[i] = -inf;  // NaN: masked
      top = fmaxf(top, x[i]);
    }
    float score[NV];
    float total = 1.f;
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
      total = sum;
      if (total > 0.f)
#pragma unroll
        for (int i = 0; i < NV; ++i) score[i] = score[i] / total;
    }
    uint32_t key[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 32 * i;
      float r = x[i];
      if (p.bias != nullptr && e < p.E) r = x[i] == -inf ? -inf : score[i] + p.bias[e];
      key[i] = r == r && r != -inf ? ordered(r) : kMasked;
    }
    if (p.groups > 1) {
      // lane g scores group g from shared memory
      uint32_t* const keys = group_keys[warp];
#pragma unroll
      for (int i = 0; i < NV; ++i)
        keys[lane + 32 * i] = p.bias != nullptr || key[i] == kMasked ? key[i] : ordered(score[i]);
      __syncwarp();
      const int per = p.E / p.groups;
      uint32_t gkey = kMasked;
      if (lane < p.groups) {
        uint32_t a = kMasked, b = kMasked;  // the two largest
        for (int i = 0; i < per; ++i) {
          const uint32_t k = keys[lane * per + i];
          b = max(b, min(a, k));
          a = max(a, k);
        }
        if (a != kMasked) gkey = ordered(b != kMasked ? from_ordered(a) + from_ordered(b) : from_ordered(a));
      }
      __syncwarp();
      uint32_t open = 0;  // bit g: group g stays
      for (int j = 0; j < p.top_groups; ++j) {
        const uint32_t best = __reduce_max_sync(0xffffffffu, gkey);
        if (best == kMasked) break;
        const uint32_t who = __ballot_sync(0xffffffffu, gkey == best);
        const int g = __ffs((int)who) - 1;
        open |= 1u << g;
        if (lane == g) gkey = kMasked;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        if (e < p.E && !((open >> (e / per)) & 1u)) key[i] = kMasked;
      }
    }
    // the top k, best first; lane j keeps the j-th
    int my_id = -1;
    float my_score = 0.f;
    for (int j = 0; j < p.k; ++j) {
      uint32_t best = kMasked;
#pragma unroll
      for (int i = 0; i < NV; ++i) best = max(best, key[i]);
      const uint32_t all = __reduce_max_sync(0xffffffffu, best);
      if (all == kMasked) break;
      uint32_t e = 0xffffffffu;
#pragma unroll
      for (int i = NV - 1; i >= 0; --i)
        if (key[i] == all) e = (uint32_t)(lane + 32 * i);
      e = __reduce_min_sync(0xffffffffu, e);
      float mine = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if ((uint32_t)(lane + 32 * i) == e) {
          key[i] = kMasked;
          mine = score[i];
        }
      mine = __shfl_sync(0xffffffffu, mine, (int)(e & 31u));
      if (lane == j) {
        my_id = (int)e;
        my_score = mine;
      }
    }
    float w = my_score;
    if (p.renormalize) {
      float sum = w;
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      w = sum > 0.f ? w / sum : 0.f;
    }
    if (lane < p.k) {
      p.ids[t * p.k + lane] = my_id;
      p.weights[t * p.k + lane] = w * p.scale;
    }
  }
}

template <int DT>
void (*route_for(int E))(const RouteParams) {
  if (E <= 32) return route_kernel<1, DT>;
  if (E <= 64) return route_kernel<2, DT>;
  if (E <= 128) return route_kernel<4, DT>;
  if (E <= 256) return route_kernel<8, DT>;
  if (E <= 512) return route_kernel<16, DT>;
  return route_kernel<32, DT>;
}

}  // namespace

cudaError_t launch_route(const RouteParams& p, int dtype, int sms, cudaStream_t stream) {
  auto kern = dtype == kF32 ? route_for<kF32>(p.E) : dtype == kBF16 ? route_for<kBF16>(p.E) : route_for<kF16>(p.E);
  const int64_t warps = kRouteThreads / 32;
  int64_t ctas = (p.T + warps - 1) / warps;
  if (ctas > 64ll * sms) ctas = 64ll * sms;
  return launch_pdl(kern, dim3((unsigned)ctas), dim3(kRouteThreads), 0, stream, p);
}

}  // namespace nvfp4
