// NVFP4 quantisation of one 16-element block, shared by the quantise kernel
// and by the product kernels' quantising epilogue (sm_103a).
//
// For the scaled values y of a block:
//   s    = E4M3(max|y| / 6), to nearest even, at most 448
//   code = E2M1(y / s),      to nearest even, at most 6 in magnitude
// A block whose s is 0 (all |y| below 6 * 2^-10) has zero codes; a block with an
// infinity or a NaN has the scale code 0x7F (NaN) and zero codes, so a product
// over it is NaN instead of silently wrong.
#pragma once
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace nvfp4 {

// x / d rounded to nearest, given r = 1/d rounded to nearest: the product x*r is
// within an ulp, and one step with its exact residual makes it the correctly
// rounded quotient (Markstein 1990).
__device__ __forceinline__ float divide_by(float x, float minus_d, float r) {
  const float q = x * r;
  return fmaf(fmaf(q, minus_d, x), r, q);
}

// 1/s rounded to nearest for an E4M3 value s > 0: the hardware's approximation
// with one Newton step (tested for every s).
__device__ __forceinline__ float scale_reciprocal(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return fmaf(fmaf(-s, r, 1.0f), r, r);
}

// The scale code of a block from max|y| (not NaN), and the scale's value.
__device__ __forceinline__ uint32_t block_scale_code(float amax, float& s) {
  // a quotient that is a tie of E4M3 is exactly that tie
  const float t = divide_by(amax, -6.0f, 1.0f / 6.0f);
  uint16_t two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.f), "f"(t));
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(two));
  s = __half2float(__ushort_as_half((unsigned short)(h2 & 0xffffu)));
  return two & 0xffu;
}

// Two fp32 values in a 64-bit register, as the two-wide instructions take them.
__device__ __forceinline__ uint64_t pack_f32x2(float x, float y) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
  return d;
}
__device__ __forceinline__ float2 unpack_f32x2(uint64_t v) {
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// Eight E2M1 codes of eight values, the first in the lowest nibble, saturating.
__device__ __forceinline__ uint32_t e2m1x8_code(const float2 (&v)[4]) {
  uint32_t out;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(out)
      : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x),
        "f"(v[3].y));
  return out;
}

// The codes of eight of a block's values (two to a register), given the block's
// scale s > 0 and r = 1/s.  divide_by for two values at once: a quotient that is a tie
// of E2M1 (y = 5 s, say) is exactly that tie, which y*r alone misses for some s.
// Quotients beyond 6 saturate in the conversion.
__device__ __forceinline__ uint32_t quantize_8(const uint64_t (&y)[4], uint64_t minus_s, uint64_t r) {
  float2 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t q = mul2(y[i], r);
    v[i] = unpack_f32x2(fma2(fma2(q, minus_s, y[i]), r, q));
  }
  return e2m1x8_code(v);
}

// max(|a|, |b|, m), NaN if any of them is.
__device__ __forceinline__ float abs_max(float m, float a, float b) {
  float d;
  asm("{\n\t.reg .f32 x, y;\n\tabs.f32 x, %1;\n\tabs.f32 y, %2;\n\tmax.NaN.f32 %0, %3, x, y;\n\t}"
      : "=f"(d)
      : "f"(a), "f"(b), "f"(m));
  return d;
}
__device__ __forceinline__ bool is_finite_max(float m) { return m < __int_as_float(0x7f800000); }

// Byte offset of scale (row, kb) in the 128x4-atom layout of one batch.
__device__ __forceinline__ int64_t atom_offset(int64_t row, int64_t kb, int64_t rest_k) {
  return ((row >> 7) * rest_k + (kb >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (kb & 3);
}

}  // namespace nvfp4
