// The experts' rows (sm_103a): a stable sort of the routed choices by expert,
// and the weighted sum of a token's expert outputs.
//
// The sort is two launches, or one up to 4096 choices: a histogram per chunk, then every
// chunk adds up the ones before it and ranks its own choices.  Both are latency up to some
// hundred thousand choices: 32768 among 64 experts 3 + 11 us beside the products' 350.  As
// every chunk reads the counts of all, it then grows with their square: among 256 experts
// 2^20 choices 43 us, 2^22 183 us, the most (2^24) 1.5 ms, or 5.7 ms among 1024, for products
// of a hundred ms and more.  The sum is one pass over the experts' outputs, bound by their
// bytes: 4096 tokens of 8 choices, M 4096 in bf16, 53 us (5.7 TB/s).
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "layer.h"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kSortWarps = kSortThreads / 32;

// A warp's choices of its CTA's chunk are consecutive, 32 at a time; within 32
// of them the ones with the same expert find each other by a match, so ranks
// follow the order of the choices and nothing depends on timing.
__device__ __forceinline__ int32_t choice(const SortParams& p, int64_t i, int64_t end) {
  if (i >= end) return -1;
  const int32_t e = p.ids[i];
  return e >= 0 && e < p.E ? e : -1;
}

// Choices per expert of each chunk.
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const SortParams p) {
  extern __shared__ int32_t hist[];  // [E]
  pdl_launch_dependents();
  for (int e = threadIdx.x; e < p.E; e += kSortThreads) hist[e] = 0;
  pdl_wait();
  __syncthreads();
  const int64_t begin = (int64_t)blockIdx.x * kSortChunk;
  const int64_t end = begin + kSortChunk < p.n ? begin + kSortChunk : p.n;
  for (int64_t i = begin + threadIdx.x; i < end; i += kSortThreads) {
    const int32_t e = choice(p, i, end);
    if (e >= 0) atomicAdd(&hist[e], 1);  // (a count: the order does not show)
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kSortThreads)
    p.chunk_counts[(int64_t)blockIdx.x * p.E + e] = hist[e];
}

// Inclusive scan over the CTA (kSortThreads values).
__device__ __forceinline__ int32_t scan_cta(int32_t v, int32_t* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int32_t o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  if (lane == 31) part[warp] = v;
  __syncthreads();
  int32_t before = 0;
  for (int w = 0; w < warp; ++w) before += part[w];
  __syncthreads();
  return v + before;
}

// Every choice's row: the expert's first row, plus the rank of the choice among
// the expert's.  With one chunk the counts come from the chunk itself (ONE).
template <bool ONE>
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const SortParams p) {
  extern __shared__ int32_t place[];  // [warps][E] offsets, then [E] counts, [E] first tile
  __shared__ int32_t part[kSortWarps];
  int32_t* const counts = place + kSortWarps * p.E;
  int32_t* const first = counts + p.E;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_launch_dependents();
  for (int i = threadIdx.x; i < kSortWarps * p.E; i += kSortThreads) place[i] = 0;
  pdl_wait();
  __syncthreads();
  const int64_t begin = (int64_t)blockIdx.x * kSortChunk;
  const int64_t end = begin + kSortChunk < p.n ? begin + kSortChunk : p.n;
  // a warp's share: consecutive choices, whole steps of 32, all warps at work
  const int share = ((int)(end - begin) + kSortThreads - 1) / kSortThreads * 32;
  const int64_t wbegin = begin + (int64_t)warp * share;
  // the warp's choices, all loads at once
  constexpr int kSteps = kSortChunk / kSortThreads;
  int32_t ids[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) ids[s] = 32 * s < share ? choice(p, wbegin + 32 * s + lane, end) : -1;
  // the warps' own counts
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    if (32 * s >= share) break;
    const int32_t e = ids[s];
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    if (e >= 0 && lane == __ffs((int)same) - 1) place[warp * p.E + e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  // before this chunk, and in all
  for (int e = threadIdx.x; e < p.E; e += kSortThreads) {
    int32_t all = 0, before = 0;
    if (ONE) {
      for (int w = 0; w < kSortWarps; ++w) all += place[w * p.E + e];
    } else {
      const int chunks = (int)gridDim.x;
      for (int c = 0; c < chunks; ++c) {
        if (c == (int)blockIdx.x) before = all;
        all += p.chunk_counts[(int64_t)c * p.E + e];
      }
    }
    counts[e] = all;
    for (int w = 0; w < kSortWarps; ++w) {
      const int32_t own = place[w * p.E + e];
      place[w * p.E + e] = before;
      before += own;
    }
  }
  __syncthreads();
  // tiles before each expert
  int32_t carry = 0;
  for (int e0 = 0; e0 < p.E; e0 += kSortThreads) {
    const int e = e0 + (int)threadIdx.x;
    const int32_t tiles = e < p.E ? (counts[e] + p.tile_rows - 1) / p.tile_rows : 0;
    const int32_t up_to = scan_cta(tiles, part) + carry;
    if (e < p.E) first[e] = up_to - tiles;
    if (threadIdx.x == kSortThreads - 1) part[0] = up_to;
    __syncthreads();
    carry = part[0];
    __syncthreads();
  }
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) *p.tile_count = carry;
    for (int e = threadIdx.x; e < p.E; e += kSortThreads) {
      p.counts[e] = counts[e];
      p.starts[e] = first[e] * p.pitch;
      for (int i = 0, left = counts[e]; left > 0; ++i, left -= p.tile_rows)
        p.tiles[first[e] + i] = make_int4(e, (first[e] + i) * p.pitch, min(left, p.tile_rows), 0);
    }
  }
  // the choices' rows
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    if (32 * s >= share) break;
    const int64_t i = wbegin + 32 * s + lane;
    const int32_t e = ids[s];
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    if (i < end) {
      int32_t row = -1;
      if (e >= 0) {
        const int32_t rank = place[warp * p.E + e] + __popc(same & ((1u << lane) - 1u));
        const int32_t tile = rank / p.tile_rows;
        row = (first[e] + tile) * p.pitch + rank - tile * p.tile_rows;
      }
      p.rows[i] = row;
    }
    __syncwarp();
    if (e >= 0 && lane == __ffs((int)same) - 1) place[warp * p.E + e] += __popc(same);
    __syncwarp();
  }
}

// Eight consecutive values.
__device__ __forceinline__ void load_eight(const float* src, float2 (&v)[4]) {
  const float4 a = reinterpret_cast<const float4*>(src)[0], b = reinterpret_cast<const float4*>(src)[1];
  v[0] = make_float2(a.x, a.y);
  v[1] = make_float2(a.z, a.w);
  v[2] = make_float2(b.x, b.y);
  v[3] = make_float2(b.z, b.w);
}
__device__ __forceinline__ float2 two_floats(uint32_t v, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
__device__ __forceinline__ float2 two_floats(uint32_t v, __nv_bfloat16) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
}
template <typename T>
__device__ __forceinline__ void load_eight(const T* src, float2 (&v)[4]) {
  const uint4 u = *reinterpret_cast<const uint4*>(src);
  v[0] = two_floats(u.x, T());
  v[1] = two_floats(u.y, T());
  v[2] = two_floats(u.z, T());
  v[3] = two_floats(u.w, T());
}
template <typename T>
__device__ __forceinline__ uint32_t two_rounded(float2 v);
template <>
__device__ __forceinline__ uint32_t two_rounded<__half>(float2 v) {
  const __half2 h = __float22half2_rn(v);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t two_rounded<__nv_bfloat16>(float2 v) {
  const __nv_bfloat162 h = __float22bfloat162_rn(v);
  return *reinterpret_cast<const uint32_t*>(&h);
}

constexpr int kCombineThreads = 256;

// out[t] = sum_j weights[t][j] * y[rows[t][j]] in fp32, in the order of j; 8
// values per thread.  M % 8 == 0.  B choices' loads go together: 4 for a few tokens,
// where their latency counts (one token: 6.2 -> 4.2 us), 1 for many (4096 tokens of 8
// choices, M 4096: 53 us, 72 with 4 at once, which reads the rows in more streams).
// SKIP: with p.skip (asked for at run time it made one token's layer 0.1 us longer).
template <typename Y, typename T, int B, bool SKIP>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const CombineParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t chunks = p.M / 8, total = p.T * chunks;
  for (int64_t i = (int64_t)blockIdx.x * kCombineThreads + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * kCombineThreads) {
    const int64_t t = i / chunks, ch = i - t * chunks;
    float2 sum[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
    const Y* const y = static_cast<const Y*>(p.y) + ch * 8;
    for (int j0 = 0; j0 < p.k; j0 += B) {
      int32_t row[B];
      float w[B];
      float2 v[B][4];
#pragma unroll
      for (int j = 0; j < B; ++j) {
        row[j] = j0 + j < p.k ? p.rows[t * p.k + j0 + j] : -1;
        if (SKIP && row[j] >= 0) row[j] -= (row[j] >> 7) * p.skip;
        w[j] = row[j] >= 0 ? p.weights[t * p.k + j0 + j] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < B; ++j)
        if (row[j] >= 0) load_eight(y + row[j] * p.M, v[j]);
#pragma unroll
      for (int j = 0; j < B; ++j) {
        if (row[j] < 0) continue;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          sum[c].x = fmaf(w[j], v[j][c].x, sum[c].x);
          sum[c].y = fmaf(w[j], v[j][c].y, sum[c].y);
        }
      }
    }
    *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + t * p.M + ch * 8) =
        make_uint4(two_rounded<T>(sum[0]), two_rounded<T>(sum[1]), two_rounded<T>(sum[2]),
                   two_rounded<T>(sum[3]));
  }
}

}  // namespace

cudaError_t launch_sort(const SortParams& p, cudaStream_t stream) {
  const int64_t chunks = (p.n + kSortChunk - 1) / kSortChunk;
  const size_t smem = sizeof(int32_t) * (size_t)p.E * (kSortWarps + 2);
  if (chunks > 1) {
    cudaError_t err = launch_pdl(sort_count_kernel, dim3((unsigned)chunks), dim3(kSortThreads),
                                 sizeof(int32_t) * (size_t)p.E, stream, p);
    if (err != cudaSuccess) return err;
  }
  constexpr size_t most = sizeof(int32_t) * (size_t)kMaxExperts * (kSortWarps + 2);
  cudaError_t err = chunks > 1 ? allow_smem<sort_place_kernel<false>>(most) : allow_smem<sort_place_kernel<true>>(most);
  if (err != cudaSuccess) return err;
  return launch_pdl(chunks > 1 ? sort_place_kernel<false> : sort_place_kernel<true>,
                    dim3((unsigned)(chunks < 1 ? 1 : chunks)), dim3(kSortThreads), smem, stream, p);
}

template <int B, bool SKIP>
void (*combine_for(int y_dtype, int dtype))(const CombineParams) {
  if (y_dtype == kF32)
    return dtype == kBF16 ? combine_kernel<float, __nv_bfloat16, B, SKIP> : combine_kernel<float, __half, B, SKIP>;
  return dtype == kBF16 ? combine_kernel<__nv_bfloat16, __nv_bfloat16, B, SKIP> : combine_kernel<__half, __half, B, SKIP>;
}

cudaError_t launch_combine(const CombineParams& p, int y_dtype, int dtype, int sms, cudaStream_t stream) {
  int64_t ctas = (p.T * (p.M / 8) + kCombineThreads - 1) / kCombineThreads;
  if (ctas > 64ll * sms) ctas = 64ll * sms;
  const bool few = ctas < sms;
  auto kern = p.skip != 0 ? (few ? combine_for<4, true>(y_dtype, dtype) : combine_for<1, true>(y_dtype, dtype))
                          : (few ? combine_for<4, false>(y_dtype, dtype) : combine_for<1, false>(y_dtype, dtype));
  return launch_pdl(kern, dim3((unsigned)ctas), dim3(kCombineThreads), 0, stream, p);
}

}  // namespace nvfp4
