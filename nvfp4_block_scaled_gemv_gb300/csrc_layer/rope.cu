// Rotary positions: pairs of a head's elements turned by an angle that grows with
// the token's position (sm_103a).
//
//   angle = position * f_i,  (a, b) -> (a cos - b sin, b cos + a sin) * factor
//
// A frequency is held as a fraction of a turn per position in 64-bit fixed point, so
// that position * f modulo a turn is one wrapping integer product, exact at any
// position (in fp32 the angle of position 10^6 would be off by up to 0.03 rad before
// the sine is taken).  The nearest quarter turn is taken off as an integer too, and what
// is left, at most an eighth of a turn, is rounded to fp32 once: an error of 2^-25 of
// that angle.
//
// One pass, bound by the bytes of x and y: 16384 tokens x 40 heads of 128 in bf16 take 54.6 us,
// 6.15 TB/s, 91% of the measured copy; 333 x 27 3.5 us and one token 2.3 us, the time of a launch
// and of a dependent load of position, table and row.  A CTA takes a few tokens: its threads first
// work out the cosines and sines of (token, pair), once for all heads, and then rotate 8
// pairs at a time, the two 16-byte halves of 16-bit pairs.
#include <cstdint>

#include "attention.h"
#include "block_io.cuh"
#include "layer.h"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kMostPairs = 512;  // cosines and sines of a CTA: its tokens times their pairs

// cos and sin of a turn's fraction in 2^-64.
__device__ __forceinline__ float2 turn(int64_t fraction) {
  const int32_t t = (int32_t)(fraction >> 32);                     // 2^-32 turns
  const int32_t quarter = (int32_t)(((uint32_t)t + (1u << 29)) >> 30);  // nearest, modulo 4
  const int32_t rest = (int32_t)((uint32_t)t - ((uint32_t)quarter << 30));  // within 2^29
  float s, c;
  sincospif((float)rest * 0x1p-31f, &s, &c);
  const float cc = (quarter & 1) ? s : c, ss = (quarter & 1) ? c : s;
  // quarters 1 and 2 have a negative cosine, 2 and 3 a negative sine
  return make_float2(((quarter + 1) & 2) ? -cc : cc, (quarter & 2) ? -ss : ss);
}

// N consecutive elements, as fp32, with loads of as many bytes as N elements have (up to 16).
template <typename T, int N>
__device__ __forceinline__ void load_n(const T* src, float (&v)[N]) {
  if constexpr (N == 1) {
    v[0] = (float)src[0];
  } else {
    constexpr int kBytes = N * (int)sizeof(T);
    uint32_t w[kBytes / 4];
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4 u = reinterpret_cast<const uint4*>(src)[i];
        w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
      }
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(src);
      w[0] = u.x, w[1] = u.y;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (sizeof(T) == 4) {
        v[i] = __uint_as_float(w[i]);
      } else {
        const T both[2] = {reinterpret_cast<const T*>(&w[i / 2])[0], reinterpret_cast<const T*>(&w[i / 2])[1]};
        v[i] = (float)both[i & 1];
      }
    }
  }
}
template <typename T, int N>
__device__ __forceinline__ void store_n(T* dst, const float (&v)[N]) {
  if constexpr (N == 1) {
    dst[0] = from_float<T>(v[0]);
  } else {
    constexpr int kBytes = N * (int)sizeof(T);
    uint32_t w[kBytes / 4];
#pragma unroll
    for (int i = 0; i < kBytes / 4; ++i) {
      if constexpr (sizeof(T) == 4)
        w[i] = __float_as_uint(v[i]);
      else
        w[i] = pack_two(make_float2(v[2 * i], v[2 * i + 1]), T());
    }
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        reinterpret_cast<uint4*>(dst)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else {
      *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    }
  }
}

// V pairs per item (8, 4 or 1), interleaved or in two halves.  A head's items: its pairs
// V at a time, then, if they are to be copied, the elements past the pairs 2 V at a time.
template <typename T, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  __shared__ float2 turns[kMostPairs];
  pdl_launch_dependents();
  pdl_wait();
  const int t0 = (int)blockIdx.x * p.tokens_per_cta;
  const int tokens = min(p.tokens_per_cta, p.T - t0);
  for (int i = threadIdx.x; i < tokens * p.pairs; i += kThreads) {
    const int t = i / p.pairs, pair = i - t * p.pairs;
    const uint64_t f = (uint64_t)ld_now(p.table + pair);
    const int64_t pos = ld_now(p.positions + t0 + t);
    float2 cs = turn((int64_t)((uint64_t)pos * f));
    cs.x *= p.factor;
    cs.y *= p.inverse ? -p.factor : p.factor;
    turns[i] = cs;
  }
  __syncthreads();
  const int turned = p.pairs / V;
  for (int i = threadIdx.x; i < tokens * p.H * p.items; i += kThreads) {
    const int row = i / p.items, item = i - row * p.items;
    const int t = row / p.H, h = row - t * p.H;
    const T* const x = static_cast<const T*>(p.x) + (int64_t)(t0 + t) * p.x_token + (int64_t)h * p.x_head;
    T* const y = static_cast<T*>(p.y) + (int64_t)(t0 + t) * p.y_token + (int64_t)h * p.y_head;
    if (item >= turned) {
      const int at = 2 * p.pairs + 2 * V * (item - turned);
      float v[V];
      load_n<T, V>(x + at, v);
      store_n<T, V>(y + at, v);
      if (at + V < p.D) {  // (a last item may be half a one)
        load_n<T, V>(x + at + V, v);
        store_n<T, V>(y + at + V, v);
      }
      continue;
    }
    const float2* const cs = turns + t * p.pairs + V * item;
    const int first = INTERLEAVED ? 2 * V * item : V * item;
    const int second = INTERLEAVED ? first + V : first + p.pairs;
    float u[V], w[V], out_u[V], out_w[V];
    load_n<T, V>(x + first, u);
    load_n<T, V>(x + second, w);
    if constexpr (INTERLEAVED) {
      if constexpr (V == 1) {
        out_u[0] = u[0] * cs[0].x - w[0] * cs[0].y;
        out_w[0] = w[0] * cs[0].x + u[0] * cs[0].y;
      } else {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          const float2 c = cs[j], d = cs[V / 2 + j];
          out_u[2 * j] = u[2 * j] * c.x - u[2 * j + 1] * c.y;
          out_u[2 * j + 1] = u[2 * j + 1] * c.x + u[2 * j] * c.y;
          out_w[2 * j] = w[2 * j] * d.x - w[2 * j + 1] * d.y;
          out_w[2 * j + 1] = w[2 * j + 1] * d.x + w[2 * j] * d.y;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float2 c = cs[j];
        out_u[j] = u[j] * c.x - w[j] * c.y;
        out_w[j] = w[j] * c.x + u[j] * c.y;
      }
    }
    store_n<T, V>(y + first, out_u);
    store_n<T, V>(y + second, out_w);
  }
}

template <typename T>
void (*rope_for(int v, bool interleaved))(const RopeParams) {
  if (interleaved) return v == 8 ? rope_kernel<T, 8, true> : v == 4 ? rope_kernel<T, 4, true> : rope_kernel<T, 1, true>;
  return v == 8 ? rope_kernel<T, 8, false> : v == 4 ? rope_kernel<T, 4, false> : rope_kernel<T, 1, false>;
}

}  // namespace

cudaError_t launch_rope(RopeParams p, int dtype, int sms, cudaStream_t stream) {
  // The widest items that the pairs, the rest of the head and the rows' alignment allow (a
  // load is at most 16 bytes).
  const int64_t size = dtype == kF32 ? 4 : 2;
  const uint64_t bits = (uint64_t)reinterpret_cast<uintptr_t>(p.x) | (uint64_t)reinterpret_cast<uintptr_t>(p.y) |
                        (uint64_t)((p.x_token | p.x_head | p.y_token | p.y_head) * size);
  int v = 1;
  for (const int want : {8, 4})
    if (v == 1 && p.pairs % want == 0 && p.D % want == 0 && bits % (uint64_t)(want * size < 16 ? want * size : 16) == 0)
      v = want;
  const int rest = p.D - 2 * p.pairs;
  p.items = p.pairs / v + (p.copy_rest ? (rest + 2 * v - 1) / (2 * v) : 0);
  // tokens per CTA: all its cosines fit, and there are CTAs for every SM's 2048 threads
  int64_t most = kMostPairs / p.pairs;
  const int64_t fill = ((int64_t)p.T + sms * 8 - 1) / (sms * 8);
  p.tokens_per_cta = (int32_t)(fill < most ? fill : most);
  auto kern = dtype == kF32    ? rope_for<float>(v, p.interleaved)
              : dtype == kBF16 ? rope_for<__nv_bfloat16>(v, p.interleaved)
                               : rope_for<__half>(v, p.interleaved);
  const int64_t ctas = ((int64_t)p.T + p.tokens_per_cta - 1) / p.tokens_per_cta;
  return launch_pdl(kern, dim3((unsigned)ctas), dim3(kThreads), 0, stream, p);
}

}  // namespace nvfp4
