// C ABI of the operators of attention: argument validation and launches.
#include <atomic>
#include <cmath>
#include <cstdint>

#include "attention.h"
#include "internal.h"
#include "layer.h"
#include "nvfp4_gemv.h"

using namespace nvfp4;

namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int64_t kMaxBatch = int64_t(1) << 20;
constexpr int64_t kMaxPage = int64_t(1) << 20;
constexpr int64_t kMaxCache = int64_t(1) << 48;  // elements of K, or of V
constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 256;  // of a sequence: ends of tiles stay in 32 bits
constexpr int64_t kMaxPairs = 512;
// Sequences of more columns (query tokens x heads of a group) go to the kernel for prompts, which
// takes 128 or 256 rows at once; fewer take passes of 16 (heads of 64: 32) columns over the cache.  One limit for a
// head size, between where few sequences and where many of them change over.  16 sequences of 8192 tokens, us, passes
// against prompts: heads of 128: 36 columns 124 and 112, 64 columns 160 and 113 (one sequence: 21 and 30, 24 and
// 30); heads of 64: 64 columns 84 and 93; heads of 256: 32 columns 94 and 161, 64 columns 176 and 164.
int64_t few_columns_for(int64_t D) { return D == 64 ? 64 : 48; }

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

nvfp4_status_t result(cudaError_t err) {
  if (err == cudaSuccess) return NVFP4_OK;
  record_cuda_error(err);
  return NVFP4_ERR_CUDA;
}

// Multiprocessors of the current device, cached per device.
cudaError_t device_sms(int* out) {
  constexpr int kMaxDevices = 128;
  static std::atomic<int> cached[kMaxDevices];
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n <= 0) {
    err = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess) return err;
    cached[dev].store(n, std::memory_order_relaxed);
  }
  *out = n;
  return cudaSuccess;
}

bool valid_dtype(int t) { return t == NVFP4_DTYPE_FP16 || t == NVFP4_DTYPE_BF16 || t == NVFP4_DTYPE_FP32; }
uintptr_t dtype_size(int t) { return t == NVFP4_DTYPE_FP32 ? 4 : 2; }
bool valid_stride(int64_t s) { return s >= 0 && s <= kMaxStride; }
bool cached_head(int64_t D) { return D == 64 || D == 128 || D == 256; }

nvfp4_status_t validate_cache(int64_t pages, int64_t heads, int64_t D, int64_t page_size) {
  if (pages < 0 || heads < 1 || D < 1 || page_size < 1) return NVFP4_ERR_INVALID_VALUE;
  if (!cached_head(D) || page_size % kGranuleTokens != 0 || page_size > kMaxPage || pages > kMaxDim ||
      heads > 65535 || (pages > 0 && page_size * heads * D > kMaxCache / pages))
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  return NVFP4_OK;
}

nvfp4_status_t cache_call(const nvfp4_kv_rows_t* rows, int dtype, int64_t T, int64_t heads, int64_t D,
                          const int64_t* slots, const void* cache, int64_t pages, int64_t page_size,
                          bool writes, CacheParams& p) {
  const nvfp4_status_t st = validate_cache(pages, heads, D, page_size);
  if (st != NVFP4_OK) return st;
  if (!valid_dtype(dtype) || T < 0 || rows == nullptr) return NVFP4_ERR_INVALID_VALUE;
  if (!valid_stride(rows->k_token_stride) || !valid_stride(rows->k_head_stride) ||
      !valid_stride(rows->v_token_stride) || !valid_stride(rows->v_head_stride))
    return NVFP4_ERR_INVALID_VALUE;
  if (T > kMaxDim - 8) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return NVFP4_OK;
  const bool some = rows->k != nullptr || rows->v != nullptr, both = rows->k != nullptr && rows->v != nullptr;
  if (slots == nullptr || (pages > 0 && cache == nullptr) || (writes ? !both : !some)) return NVFP4_ERR_INVALID_VALUE;
  if (!aligned(rows->k, dtype_size(dtype)) || !aligned(rows->v, dtype_size(dtype)) || !aligned(slots, 8) ||
      !aligned(cache, 16) || !aligned(rows->encode_k, 4) || !aligned(rows->encode_v, 4))
    return NVFP4_ERR_MISALIGNED;
  p.cache = static_cast<uint8_t*>(const_cast<void*>(cache));
  p.slots = slots;
  p.k = rows->k;
  p.v = rows->v;
  p.encode_k = rows->encode_k;
  p.encode_v = rows->encode_v;
  p.k_head = rows->k_head_stride ? rows->k_head_stride : D;
  p.v_head = rows->v_head_stride ? rows->v_head_stride : D;
  p.k_token = rows->k_token_stride ? rows->k_token_stride : heads * D;
  p.v_token = rows->v_token_stride ? rows->v_token_stride : heads * D;
  p.capacity = pages * page_size;
  p.T = (int32_t)T;
  p.heads = (int32_t)heads;
  p.planes = (int32_t)(D / 64);
  p.page_size = (int32_t)page_size;
  p.granules = (int32_t)(page_size / kGranuleTokens);
  return NVFP4_OK;
}

// The sizes of an attention call; most_q: query tokens of a sequence, at most.
nvfp4_status_t validate_attention(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t pages,
                                  int64_t page_size, int64_t max_pages, bool ragged, int64_t max_q,
                                  int64_t* most_q) {
  const nvfp4_status_t st = validate_cache(pages, Hkv, D, page_size);
  if (st != NVFP4_OK) return st;
  if (T < 0 || B < 0 || Hq < 1 || max_pages < 0 || max_q < 0 || max_q > T) return NVFP4_ERR_INVALID_VALUE;
  if (Hq % Hkv != 0 || B > kMaxBatch || T > kMaxDim / Hq || max_pages > kMaxTokens / page_size)
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!ragged && ((B == 0 && T != 0) || (B != 0 && (T % B != 0 || (max_q != 0 && max_q != T / B)))))
    return NVFP4_ERR_INVALID_VALUE;
  *most_q = !ragged ? (B == 0 ? 0 : T / B) : max_q != 0 ? max_q : T;
  // tiles of the kernel for few query tokens, over sequences, heads and passes, are counted in 32 bits
  const int64_t columns = *most_q * (Hq / Hkv) < few_columns_for(D) ? *most_q * (Hq / Hkv) : few_columns_for(D);
  const int64_t passes = (columns + 7) / 8;
  if (B * Hkv * (passes > 0 ? passes : 1) > kMaxDim / (max_pages * page_size / 32 + 1)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  return NVFP4_OK;
}

// Columns of a pass of the kernel for few query tokens.  Beside prompts sequences are taken to have a
// single token (heads of 128, 4 heads a group, 4 prompts of 512 on 2000 tokens and 64 sequences of one token: 125 us
// with passes of 8 columns, 137 with 16; 64 of 4 tokens: 149 and 138; a prompt of 2048 and 4096 of one token: 210
// and 296).
int few_pass(const AttentionParams& p, int64_t D, int64_t columns) {
  const int64_t expected = columns <= few_columns_for(D) ? columns : p.group;
  return attention_columns((int)D, expected < p.few_columns ? expected : p.few_columns);
}

// The sizes that both kernels work from; with few_columns: sequences of more columns are the
// prompt kernel's, or, if none are to be expected, left out.
AttentionParams sizes_of(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t page_size,
                         int64_t max_pages, int64_t columns, bool ragged) {
  AttentionParams p = {};
  p.ragged = ragged;
  p.T = (int32_t)T;
  p.B = (int32_t)B;
  p.Hq = (int32_t)Hq;
  p.Hkv = (int32_t)Hkv;
  p.group = (int32_t)(Hq / Hkv);
  p.max_pages = (int32_t)max_pages;
  p.granules = (int32_t)(page_size / kGranuleTokens);
  p.capacity = max_pages * page_size;
  p.most_columns = (int32_t)columns;
  p.few_columns = (int32_t)(columns < few_columns_for(D) ? columns : few_columns_for(D));
  return p;
}

// The kernels of a call use the workspace one after another.
int64_t workspace_for(const AttentionParams& p, int64_t D, int64_t columns) {
  const int64_t few = p.ragged || columns <= few_columns_for(D) ? attention_workspace((int)D, few_pass(p, D, columns)) : 0;
  const int64_t prompt = columns > few_columns_for(D) ? attention_prompt_workspace(p, (int)D) : 0;
  return few > prompt ? few : prompt;
}

}  // namespace

extern "C" {

nvfp4_status_t nvfp4_rope(const void* x, int dtype, int64_t T, int64_t H, int64_t D, const int32_t* positions,
                          const int64_t* table, int64_t pairs, const nvfp4_rope_options_t* options, void* y,
                          struct CUstream_st* stream) {
  static const nvfp4_rope_options_t kDefaults = {0, 0, 1.0f, 0, 0, 0, 0};
  const nvfp4_rope_options_t& opt = options ? *options : kDefaults;
  if (!valid_dtype(dtype) || T < 0 || H < 0 || D < 0 || pairs < 0 || (opt.interleaved != 0 && opt.interleaved != 1) ||
      (opt.inverse != 0 && opt.inverse != 1) || !std::isfinite(opt.factor) || !valid_stride(opt.x_token_stride) ||
      !valid_stride(opt.x_head_stride) || !valid_stride(opt.y_token_stride) || !valid_stride(opt.y_head_stride))
    return NVFP4_ERR_INVALID_VALUE;
  if (2 * pairs > D) return NVFP4_ERR_INVALID_VALUE;
  if (pairs < 1 || pairs > kMaxPairs || T > kMaxDim || D > 65536 || H > 65536 || H * D > kMaxDim) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (T == 0 || H == 0) return NVFP4_OK;
  if (x == nullptr || y == nullptr || positions == nullptr || table == nullptr) return NVFP4_ERR_INVALID_VALUE;
  if (!aligned(x, dtype_size(dtype)) || !aligned(y, dtype_size(dtype)) || !aligned(positions, 4) || !aligned(table, 8))
    return NVFP4_ERR_MISALIGNED;
  RopeParams p = {};
  p.x = x;
  p.y = y;
  p.positions = positions;
  p.table = table;
  p.x_head = opt.x_head_stride ? opt.x_head_stride : D;
  p.y_head = opt.y_head_stride ? opt.y_head_stride : D;
  p.x_token = opt.x_token_stride ? opt.x_token_stride : H * D;
  p.y_token = opt.y_token_stride ? opt.y_token_stride : H * D;
  // in place: every element is written by the thread that read it, if it has one place
  if (x == y && (p.x_head != p.y_head || p.x_token != p.y_token)) return NVFP4_ERR_INVALID_VALUE;
  p.T = (int32_t)T;
  p.H = (int32_t)H;
  p.D = (int32_t)D;
  p.pairs = (int32_t)pairs;
  p.interleaved = opt.interleaved;
  p.inverse = opt.inverse;
  p.factor = opt.factor;
  p.copy_rest = x != y;
  int sms = 0;
  const cudaError_t err = device_sms(&sms);
  if (err != cudaSuccess) return result(err);
  return result(launch_rope(p, dtype, sms, (cudaStream_t)stream));
}

size_t nvfp4_kv_cache_bytes(int64_t pages, int64_t heads, int64_t D, int64_t page_size) {
  if (validate_cache(pages, heads, D, page_size) != NVFP4_OK) return 0;
  return (size_t)pages * (size_t)(page_size / kGranuleTokens * heads * 2 * (D / 64) * kPlaneBytes);
}

nvfp4_status_t nvfp4_kv_write(const nvfp4_kv_rows_t* rows, int dtype, int64_t T, int64_t heads, int64_t D,
                              const int64_t* slots, void* cache, int64_t pages, int64_t page_size,
                              struct CUstream_st* stream) {
  CacheParams p = {};
  const nvfp4_status_t st = cache_call(rows, dtype, T, heads, D, slots, cache, pages, page_size, true, p);
  if (st != NVFP4_OK || T == 0) return st;
  return result(launch_kv_write(p, dtype, (cudaStream_t)stream));
}

nvfp4_status_t nvfp4_kv_read(const nvfp4_kv_rows_t* rows, int dtype, int64_t T, int64_t heads, int64_t D,
                             const int64_t* slots, const void* cache, int64_t pages, int64_t page_size,
                             struct CUstream_st* stream) {
  CacheParams p = {};
  const nvfp4_status_t st = cache_call(rows, dtype, T, heads, D, slots, cache, pages, page_size, false, p);
  if (st != NVFP4_OK || T == 0) return st;
  return result(launch_kv_read(p, dtype, (cudaStream_t)stream));
}

size_t nvfp4_attention_workspace_bytes(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t page_size,
                                       int64_t max_pages, int ragged, int64_t max_q) {
  int64_t most_q = 0;
  if (validate_attention(T, B, Hq, Hkv, D, 0, page_size, max_pages, ragged != 0, max_q, &most_q) != NVFP4_OK) return 0;
  if (T == 0) return 0;
  const int64_t columns = most_q * (Hq / Hkv);
  const int64_t bytes = workspace_for(sizes_of(T, B, Hq, Hkv, D, page_size, max_pages, columns, ragged != 0), D, columns);
  return (size_t)(bytes > 256 ? bytes : 256);
}

nvfp4_status_t nvfp4_attention(const void* q, int dtype, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                               const void* cache, int64_t pages, int64_t page_size, const int32_t* page_table,
                               int64_t max_pages, const int32_t* lengths, int64_t B,
                               const nvfp4_attention_options_t* options, void* out, void* workspace,
                               size_t workspace_bytes, struct CUstream_st* stream) {
  static const nvfp4_attention_options_t kDefaults = {0.0f, 1, 0, 0, nullptr, nullptr, nullptr, nullptr, 0, 0};
  const nvfp4_attention_options_t& opt = options ? *options : kDefaults;
  int64_t most_q = 0;
  const nvfp4_status_t st =
      validate_attention(T, B, Hq, Hkv, D, pages, page_size, max_pages, opt.q_starts != nullptr, opt.max_q, &most_q);
  if (st != NVFP4_OK) return st;
  if ((dtype != NVFP4_DTYPE_FP16 && dtype != NVFP4_DTYPE_BF16) || !(opt.scale >= 0.f) || !std::isfinite(opt.scale) ||
      (opt.causal != 0 && opt.causal != 1) || opt.window < 0 || (opt.window > 0 && opt.causal == 0) ||
      !valid_stride(opt.q_token_stride) || !valid_stride(opt.q_head_stride))
    return NVFP4_ERR_INVALID_VALUE;
  if (T == 0 || B == 0) return NVFP4_OK;
  const int64_t columns = most_q * (Hq / Hkv);
  AttentionParams p = sizes_of(T, B, Hq, Hkv, D, page_size, max_pages, columns, opt.q_starts != nullptr);
  const size_t need = (size_t)workspace_for(p, D, columns);
  if (q == nullptr || out == nullptr || lengths == nullptr || (max_pages > 0 && page_table == nullptr) ||
      (pages > 0 && cache == nullptr) || workspace == nullptr || workspace_bytes < need)
    return NVFP4_ERR_INVALID_VALUE;
  const int64_t head_stride = opt.q_head_stride ? opt.q_head_stride : D;
  const int64_t token_stride = opt.q_token_stride ? opt.q_token_stride : Hq * D;
  if (!aligned(q, 16) || head_stride % 8 != 0 || token_stride % 8 != 0 || !aligned(out, 16) || !aligned(cache, 16) ||
      !aligned(workspace, 256) || !aligned(page_table, 4) || !aligned(lengths, 4) || !aligned(opt.q_starts, 4) ||
      !aligned(opt.encode_k, 4) || !aligned(opt.encode_v, 4) || !aligned(opt.lse, 4))
    return NVFP4_ERR_MISALIGNED;
  p.q = q;
  p.out = out;
  p.lse = opt.lse;
  p.cache = static_cast<const uint8_t*>(cache);
  p.page_table = page_table;
  p.lengths = lengths;
  p.q_starts = opt.q_starts;
  p.encode_k = opt.encode_k;
  p.encode_v = opt.encode_v;
  p.q_token = token_stride;
  p.q_head = head_stride;
  p.pages = pages;
  p.uniform_n = opt.q_starts ? 0 : (int32_t)(T / B);
  p.window = opt.window;
  p.causal = opt.causal;
  p.bf16 = dtype == NVFP4_DTYPE_BF16;
  const double scale = opt.scale > 0.f ? (double)opt.scale : 1.0 / std::sqrt((double)D);
  p.scale_log2 = (float)(scale * 1.4426950408889634);
  int sms = 0;
  const cudaError_t err = device_sms(&sms);
  if (err != cudaSuccess) return result(err);
  if (columns > few_columns_for(D)) {
    const cudaError_t ran = launch_attention_prompt(p, (int)D, workspace, (cudaStream_t)stream);
    if (ran != cudaSuccess || opt.q_starts == nullptr) return result(ran);
  }
  return result(launch_attention(p, (int)D, few_pass(p, D, columns), workspace, sms, (cudaStream_t)stream));
}

}  // extern "C"
