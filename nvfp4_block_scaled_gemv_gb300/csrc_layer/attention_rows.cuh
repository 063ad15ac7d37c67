// What both kernels of attention (attention.cu, attention_prompt.cu) take a row of queries for: which rows
// a sequence has, what a row sees, and the arithmetic of its softmax.
#pragma once
#include <cstdint>

#include "attention.h"
#include "ptx.cuh"

namespace nvfp4 {

// A sequence's query tokens: rows of q from q0, n of them.
struct QueryRows {
  int32_t q0, n;
};
__device__ __forceinline__ QueryRows query_rows(const AttentionParams& p, int b) {
  if (p.q_starts == nullptr) return {b * p.uniform_n, p.uniform_n};
  const int32_t from = max(ld_now(p.q_starts + b), 0), to = min(ld_now(p.q_starts + b + 1), p.T);
  return {from, max(to - from, 0)};
}

// Its cached tokens, no more than the page table has room for.
__device__ __forceinline__ int32_t cached_tokens(const AttentionParams& p, int b, bool& beyond) {
  const int32_t length = ld_now(p.lengths + b);
  beyond = (int64_t)length > p.capacity;
  return beyond ? (int32_t)p.capacity : max(length, 0);
}

// The tokens [lo, hi) that query token i of n sees in a sequence of that length.
__device__ __forceinline__ void token_sees(const AttentionParams& p, int32_t length, int32_t n, int32_t i, int32_t& lo,
                                           int32_t& hi) {
  lo = 0;
  hi = length;
  if (p.causal) {
    hi = length - n + i + 1;  // (0 or less: none)
    if (p.window > 0 && hi > p.window) lo = hi - p.window;
  }
}

// p of a row's reference in base 2.  Scores pass the reference by 8 at most, so that fp16 holds every p (2^15 and the
// 2^-4 above), and below its normal numbers are only p's under 2^-21 of the reference's, which are off by 2^-32 of that.
// (With the reference at 1 these were 2^-14 and 2^-25: 131071 tokens of e^-18 beside one lost a tenth of their sum.)
constexpr float kReferenceP = 7.f;

__device__ __forceinline__ float exp2_fast(float x) {
  float d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(x));
  return d;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

}  // namespace nvfp4
