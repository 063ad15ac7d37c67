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

// The scale code of a block from max|y| (not NaN), and the scale's value.
__device__ __forceinline__ uint32_t block_scale_code(float amax, float& s) {
  // the division is IEEE, so a quotient that is a tie of E4M3 stays one
  const float t = amax / 6.0f;
  uint16_t two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.f), "f"(t));
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(two));
  s = __half2float(__ushort_as_half((unsigned short)(h2 & 0xffffu)));
  return two & 0xffu;
}

// y / s rounded to nearest, for s an E4M3 value > 0 and r = 1/s rounded to
// nearest: the product y*r is within an ulp, and one step with its exact
// residual makes it the correctly rounded quotient (Markstein 1990).  A quotient
// that is a tie of E2M1 (y = 5 s, say) is therefore exactly that tie, which y*r
// alone misses for some s.
__device__ __forceinline__ float divide_by_scale(float y, float s, float r) {
  const float q = y * r;
  return fmaf(fmaf(-q, s, y), r, q);
}

// Two E2M1 codes (lo in the low nibble) of two values, saturating.
__device__ __forceinline__ uint32_t e2m1x2_code(float lo, float hi) {
  uint32_t out;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\t"
      "mov.b32 %0, {b, 0, 0, 0};\n\t}"
      : "=r"(out)
      : "f"(lo), "f"(hi));
  return out;
}

// Eight E2M1 codes of eight values, the first in the lowest nibble.
__device__ __forceinline__ uint32_t e2m1x8_code(const float (&v)[8]) {
  uint32_t out;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(out)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return out;
}

// The codes of eight of a block's values, given the block's scale s.
// Quotients beyond 6 saturate in the conversion.
__device__ __forceinline__ uint32_t quantize_8(const float (&y)[8], float s, float r) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = divide_by_scale(y[i], s, r);
  return e2m1x8_code(v);
}

// Byte offset of scale (row, kb) in the 128x4-atom layout of one batch.
__device__ __forceinline__ int64_t atom_offset(int64_t row, int64_t kb, int64_t rest_k) {
  return ((row >> 7) * rest_k + (kb >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (kb & 3);
}

}  // namespace nvfp4
