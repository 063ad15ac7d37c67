// A block of 16 values as it is in memory, its loads, and its way to codes and
// back: shared by the kernels that quantise and dequantise (quantize.cu, kv_cache.cu).
#pragma once
#include <cstdint>

#include "ptx.cuh"
#include "quantize.cuh"

namespace nvfp4 {

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// 16 consecutive values as they are in memory.
template <typename T>
struct RawBlock {
  static constexpr int kWords = 4 * (int)sizeof(T);
  uint32_t w[kWords];
};

// With 32-byte loads (ALIGN 32), 16-byte loads (16) or one by one (1).
template <typename T, int ALIGN>
__device__ __forceinline__ void load_raw(const T* src, RawBlock<T>& b) {
  if constexpr (ALIGN == 1) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 16; ++i) b.w[i] = reinterpret_cast<const uint32_t*>(src)[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        b.w[i] = (uint32_t)reinterpret_cast<const uint16_t*>(src)[2 * i] |
                 (uint32_t)reinterpret_cast<const uint16_t*>(src)[2 * i + 1] << 16;
    }
  } else {
#pragma unroll
    for (int i = 0; i < RawBlock<T>::kWords; i += 8) {
      const uint32_t* const at = reinterpret_cast<const uint32_t*>(src) + i;
      uint32_t v[8];
      if constexpr (ALIGN == 32) {
        ld_stream_now_256(at, v);
      } else {
        const uint4 a = ld_now(reinterpret_cast<const uint4*>(at)), c = ld_now(reinterpret_cast<const uint4*>(at + 4));
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = c.x, v[5] = c.y, v[6] = c.z, v[7] = c.w;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) b.w[i + j] = v[j];
    }
  }
}

__device__ __forceinline__ uint32_t abs_max_word(uint32_t a, uint32_t b, float) {
  return __float_as_uint(abs_max(0.f, __uint_as_float(a), __uint_as_float(b)));
}
__device__ __forceinline__ uint32_t abs_max_word(uint32_t a, uint32_t b, __half) {
  uint32_t d;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a & 0x7fff7fffu), "r"(b & 0x7fff7fffu));
  return d;
}
__device__ __forceinline__ uint32_t abs_max_word(uint32_t a, uint32_t b, __nv_bfloat16) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a & 0x7fff7fffu), "r"(b & 0x7fff7fffu));
  return d;
}
// Values 2i and 2i+1 of a block.
__device__ __forceinline__ float2 two_of(const RawBlock<float>& b, int i) {
  return make_float2(__uint_as_float(b.w[2 * i]), __uint_as_float(b.w[2 * i + 1]));
}
__device__ __forceinline__ float2 two_of(const RawBlock<__half>& b, int i) {
  return __half22float2(*reinterpret_cast<const __half2*>(&b.w[i]));
}
__device__ __forceinline__ float2 two_of(const RawBlock<__nv_bfloat16>& b, int i) {
  return make_float2(__uint_as_float(b.w[i] << 16), __uint_as_float(b.w[i] & 0xffff0000u));
}

// max|x| of a block, NaN if it holds one.
template <typename T>
__device__ __forceinline__ float raw_abs_max(const RawBlock<T>& b) {
  constexpr int n = RawBlock<T>::kWords;
  uint32_t m[n / 2];
#pragma unroll
  for (int i = 0; i < n / 2; ++i) m[i] = abs_max_word(b.w[2 * i], b.w[2 * i + 1], T());
#pragma unroll
  for (int d = n / 4; d; d /= 2)
#pragma unroll
    for (int i = 0; i < d; ++i) m[i] = abs_max_word(m[i], m[i + d], T());
  if constexpr (sizeof(T) == 4) {
    return __uint_as_float(m[0]);
  } else {
    RawBlock<T> last;
    last.w[0] = m[0];
    const float2 v = two_of(last, 0);
    return abs_max(0.f, v.x, v.y);
  }
}

// A block's codes and scale code.  (Rounding is monotone, so max|y| is the
// rounded product of max|x|.)
template <typename T>
__device__ __forceinline__ uint32_t quantize_block(const RawBlock<T>& b, float encode, uint2& q) {
  const float amax = raw_abs_max(b) * encode;
  q = make_uint2(0u, 0u);
  if (!is_finite_max(amax)) return 0x7Fu;
  float s;
  const uint32_t code = block_scale_code(amax, s);
  if (s > 0.f) {
    const float r = scale_reciprocal(s);
    const uint64_t r2 = pack_f32x2(r, r), s2 = pack_f32x2(-s, -s), e2 = pack_f32x2(encode, encode);
    uint64_t lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = two_of(b, i), c = two_of(b, i + 4);
      lo[i] = mul2(pack_f32x2(a.x, a.y), e2);
      hi[i] = mul2(pack_f32x2(c.x, c.y), e2);
    }
    q = make_uint2(quantize_8(lo, s2, r2), quantize_8(hi, s2, r2));
  }
  return code;
}

// Two fp32 values rounded to the output type.
__device__ __forceinline__ uint32_t pack_two(float2 v, __half) {
  const __half2 h = __float22half2_rn(v);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_two(float2 v, __nv_bfloat16) {
  const __nv_bfloat162 h = __float22bfloat162_rn(v);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A block's values: code * scale has 6 significant bits and is exact in fp16; the
// product with `scale` (fp32) and the result's type round.
template <typename T, int ALIGN>
__device__ __forceinline__ void dequantize_block(uint2 q, uint32_t code, float scale, T* dst) {
  const uint32_t s2 = e4m3x2_to_f16x2(code | code << 8);
  uint32_t h[2][4];
  e2m1x8_to_f16x2x4(q.x, h[0]);
  e2m1x8_to_f16x2x4(q.y, h[1]);
  const uint64_t scale2 = pack_f32x2(scale, scale);
  float2 y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&h[i / 4][i % 4]),
                              *reinterpret_cast<const __half2*>(&s2));
    const float2 f = __half22float2(v);
    y[i] = unpack_f32x2(mul2(pack_f32x2(f.x, f.y), scale2));
  }
  if constexpr (ALIGN == 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dst[2 * i] = from_float<T>(y[i].x);
      dst[2 * i + 1] = from_float<T>(y[i].y);
    }
  } else {
    constexpr int kWords = RawBlock<T>::kWords;
    uint32_t w[kWords];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(T) == 4) {
        w[2 * i] = __float_as_uint(y[i].x);
        w[2 * i + 1] = __float_as_uint(y[i].y);
      } else {
        w[i] = pack_two(y[i], T());
      }
    }
#pragma unroll
    for (int i = 0; i < kWords; i += 8) {
      uint32_t* const to = reinterpret_cast<uint32_t*>(dst) + i;
      if constexpr (ALIGN == 32) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[i]),
                     "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]), "r"(w[i + 5]),
                     "r"(w[i + 6]), "r"(w[i + 7])
                     : "memory");
      } else {
        reinterpret_cast<uint4*>(to)[0] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
        reinterpret_cast<uint4*>(to)[1] = make_uint4(w[i + 4], w[i + 5], w[i + 6], w[i + 7]);
      }
    }
  }
}

}  // namespace nvfp4
