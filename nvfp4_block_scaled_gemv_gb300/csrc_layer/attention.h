// Host/device interface of the operators of attention: rotary positions, the
// 4-bit key and value cache, and attention on it.
#pragma once
#include <cstdint>

#include <cuda_runtime.h>

namespace nvfp4 {

// ---- rotary positions (rope.cu) ----

struct RopeParams {
  const void* x;              // [T][H][D], strides in elements
  void* y;
  const int32_t* positions;   // [T]
  const int64_t* table;       // [pairs]: 2^-64 turns per position
  int64_t x_token, x_head, y_token, y_head;
  int32_t T, H, D, pairs;     // pairs > 0; 2 * pairs <= D
  int32_t interleaved, inverse;
  int32_t copy_rest;          // 0: the elements past the pairs are in place already
  float factor;
  // set by the launcher
  int32_t tokens_per_cta, items;
};
cudaError_t launch_rope(RopeParams p, int dtype, int sms, cudaStream_t stream);

// ---- the cache (kv_cache.cu) ----

// [pages][heads][page_size/16] granules of 16 tokens; a granule holds K and then V, each
// as head_dim/64 planes of 64 elements: 16 rows of 32 bytes of codes, then 16 rows of 4
// scale bytes.  What attention reads of a head's 16 tokens is thus one run of bytes.
constexpr int kGranuleTokens = 16;
constexpr int kPlaneBytes = kGranuleTokens * 36;
constexpr int kPlaneScales = kGranuleTokens * 32;  // where a plane's scales begin

struct CacheParams {
  uint8_t* cache;
  const int64_t* slots;       // [T]: page * page_size + place in the page; others are skipped
  void* k;                    // [T][heads][D] (read: may be null)
  void* v;
  const float* encode_k;      // [heads] or null
  const float* encode_v;
  int64_t k_token, k_head, v_token, v_head;  // strides in elements
  int64_t capacity;           // slots of the cache
  int32_t T, heads, planes, page_size, granules;  // granules per page
  int64_t places;             // set by the launcher
};
cudaError_t launch_kv_write(CacheParams p, int dtype, cudaStream_t stream);
cudaError_t launch_kv_read(CacheParams p, int dtype, cudaStream_t stream);

// ---- attention (attention.cu) ----

struct AttentionParams {
  const void* q;              // [T][Hq][D], strides in elements
  void* out;                  // [T][Hq][D]
  float* lse;                 // [T][Hq] or null
  const uint8_t* cache;
  const int32_t* page_table;  // [B][max_pages]
  const int32_t* lengths;     // [B]
  const int32_t* q_starts;    // [B + 1], or null: uniform_n tokens each
  const float* encode_k;      // [Hkv] or null
  const float* encode_v;
  int64_t q_token, q_head;
  int64_t pages, capacity;    // capacity: max_pages * page_size
  int32_t T, B, Hq, Hkv, group, uniform_n, max_pages, granules, window, causal;
  int32_t most_columns;       // of a sequence (query tokens x heads of a group), at most
  int32_t few_columns;        // sequences of more columns are the prompt kernel's
  int32_t ragged;             // q_starts are given
  int32_t bf16;
  float scale_log2;           // scale * log2(e)
  // split of the work (set by the launcher)
  float* partial;             // pieces: [CTAs][2] and [CTAs][warps]
  int32_t* row_tiles;         // prompts in ragged batches: [B + 1] row tiles before each sequence
  int32_t splits;             // prompts: parts of a row tile's tokens
  int32_t units;              // prompts: row tiles x heads x parts, at most
  int4* pieces;               // [CTAs][2]: {last CTA or -1, head, first column, beyond}, {n, q0} of the item that goes on in the next
};
constexpr int kAttentionCtas = 152;  // most CTAs of a launch, which the workspace is made for
// Columns (query token and head of a group, together) that one pass over the cache takes
// for a head size and the most columns of a sequence.
int attention_columns(int D, int64_t most);
int64_t attention_workspace(int D, int columns);
cudaError_t launch_attention(AttentionParams p, int D, int columns, void* workspace, int sms, cudaStream_t stream);
// Sequences of more than p.few_columns columns (attention_prompt.cu).
cudaError_t launch_attention_prompt(const AttentionParams& p, int D, void* workspace, cudaStream_t stream);
// Bytes of its workspace, from p's sizes alone.
int64_t attention_prompt_workspace(const AttentionParams& p, int D);
cudaError_t prompt_wait_timeouts(int reset, int* out);
cudaError_t attention_wait_timeouts(int reset, int* out);

}  // namespace nvfp4
