// C ABI of the layer operators: argument validation and launches.
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>

#include "internal.h"
#include "layer.h"
#include "nvfp4_gemv.h"

using namespace nvfp4;

namespace {

constexpr int64_t kMaxK = int64_t(1) << 30;
constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxRows = int64_t(1) << 40;  // rows of all batches
constexpr int64_t kMaxChoices = int64_t(1) << 24;
constexpr int64_t kMaxMapBytes = int64_t(1) << 40;  // a tensor map's outer stride

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

nvfp4_status_t result(cudaError_t err) {
  if (err == cudaSuccess) return NVFP4_OK;
  record_cuda_error(err);
  return NVFP4_ERR_CUDA;
}

// Multiprocessors of the current device, cached per device.
cudaError_t sm_count(int* out) {
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
bool valid_activation(int a) { return a >= NVFP4_ACT_NONE && a <= NVFP4_ACT_GELU_ERF; }

nvfp4_status_t validate_rows(int dtype, int64_t rows, int64_t K, int64_t L, int64_t stride,
                             int sf_layout) {
  if (!valid_dtype(dtype) || rows < 0 || K < 0 || L < 0 || (stride != 0 && stride < K))
    return NVFP4_ERR_INVALID_VALUE;
  if (sf_layout != NVFP4_SF_PLAIN && sf_layout != NVFP4_SF_PERMUTED_128x4) return NVFP4_ERR_INVALID_VALUE;
  if (K % 16 != 0 || K > kMaxK || rows > kMaxDim || L > kMaxDim || (rows != 0 && L > kMaxRows / rows) ||
      stride > kMaxK * 16)
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  return NVFP4_OK;
}

// Tile of the experts' products and what follows from it (host arithmetic).
struct MoeShape {
  int64_t choices, tiles, rows;
  int tile_rows, pitch;
  // the plan: tiles (16 bytes each), their number, the sort's chunk counts
  int64_t count_at, chunks_at, bytes;
};

int moe_tile_rows(int64_t T, int64_t k, int64_t E) {
  // about twice an expert's even share, and no more than all tokens
  const int64_t share = 2 * ceil_div(T * k, E);
  const int64_t need = share < T ? share : T;
  return need <= 16 ? 16 : need <= 32 ? 32 : need <= 64 ? 64 : need <= 128 ? 128 : 256;
}

MoeShape moe_shape(int64_t T, int64_t k, int64_t E) {
  MoeShape s;
  s.choices = T * k;
  s.tile_rows = moe_tile_rows(T, k, E);
  s.pitch = s.tile_rows < 128 ? 128 : s.tile_rows;  // a tile starts on a scale atom
  s.tiles = s.choices / s.tile_rows + (E < s.choices ? E : s.choices);
  s.rows = s.tiles * s.pitch;
  s.count_at = s.tiles * 16;
  s.chunks_at = s.count_at + 16;
  s.bytes = s.chunks_at + ceil_div(ceil_div(s.choices, kSortChunk) * E * 4, 16) * 16;
  return s;
}

nvfp4_status_t validate_moe(int64_t T, int64_t k, int64_t E) {
  if (T < 0 || k < 1 || E < 1) return NVFP4_ERR_INVALID_VALUE;
  if (E > kMaxExperts || k > kMaxTopK || k > E || T > kMaxChoices / k) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (moe_shape(T, k, E).rows > kMaxDim) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  return NVFP4_OK;
}

// A weight matrix [G][M][K/2] that a tensor map can describe.
nvfp4_status_t validate_product(int64_t M, int64_t N, int64_t K, int64_t G) {
  if (M < 0 || N < 0 || K < 0 || G < 0) return NVFP4_ERR_INVALID_VALUE;
  if (K % 32 != 0 || K > kMaxK || M > kMaxDim || N > kMaxDim || G > kMaxDim)
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if ((M != 0 && G > kMaxRows / M) || (N != 0 && G > kMaxRows / N)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  const int64_t most = M > N ? M : N;
  if (K != 0 && most >= kMaxMapBytes / (K / 2 > 0 ? K / 2 : 1)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  return NVFP4_OK;
}

// Tiles are counted in 32 bits (the dense product's smallest have 128 x 16 outputs).
bool dense_tiles_fit(int64_t M, int64_t N, int64_t L) {
  return M == 0 || N == 0 || L <= kMaxDim / ceil_div(M, 128) / ceil_div(N, 16);
}
nvfp4_status_t validate_grouped(const MoeShape& s, int64_t M, int64_t K, int64_t E) {
  const nvfp4_status_t st = validate_product(M, s.rows, K, E);
  if (st != NVFP4_OK) return st;
  return s.tiles * ceil_div(M, 128) > kMaxDim ? NVFP4_ERR_UNSUPPORTED_SHAPE : NVFP4_OK;
}

// The sizes of the whole layer (those of its steps among them).
nvfp4_status_t validate_ffn(int64_t T, int64_t k, int64_t E, int64_t D, int64_t F) {
  nvfp4_status_t st = validate_moe(T, k, E);
  if (st != NVFP4_OK) return st;
  if (D < 0 || F < 0) return NVFP4_ERR_INVALID_VALUE;
  if (D % 32 != 0 || F % 32 != 0 || D == 0 || F == 0 || F > kMaxDim / 2) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  const MoeShape s = moe_shape(T, k, E);
  st = validate_grouped(s, 2 * F, D, E);
  return st != NVFP4_OK ? st : validate_grouped(s, D, F, E);
}

SortParams sort_params(const int32_t* ids, const MoeShape& s, int64_t E, int32_t* rows, int32_t* counts,
                       int32_t* starts, void* plan) {
  uint8_t* const base = static_cast<uint8_t*>(plan);
  SortParams p = {};
  p.ids = ids;
  p.rows = rows;
  p.counts = counts;
  p.starts = starts;
  p.tiles = reinterpret_cast<int4*>(base);
  p.tile_count = reinterpret_cast<int32_t*>(base + s.count_at);
  p.chunk_counts = reinterpret_cast<int32_t*>(base + s.chunks_at);
  p.n = s.choices;
  p.E = (int32_t)E;
  p.tile_rows = s.tile_rows;
  p.pitch = s.pitch;
  return p;
}

GemmArgs moe_gemm_args(const void* a, const void* sfa, const void* b, const void* sfb, const void* plan,
                       const MoeShape& s, int64_t E, int64_t M, int64_t K) {
  GemmArgs g = {};
  g.a = static_cast<const uint8_t*>(a);
  g.sfa = static_cast<const uint8_t*>(sfa);
  g.b = static_cast<const uint8_t*>(b);
  g.sfb = static_cast<const uint8_t*>(sfb);
  g.M = M;
  g.N = s.rows;
  g.K = K;
  g.G = E;
  g.tiles = static_cast<const int4*>(plan);
  g.tile_count = reinterpret_cast<const int32_t*>(static_cast<const uint8_t*>(plan) + s.count_at);
  g.max_tiles = s.tiles;
  g.tile_rows = s.tile_rows;
  g.alpha = 1.0f;
  g.encode = 1.0f;
  return g;
}

// An expert's output before the weighted sum is fp32, and rounded once, after the sum; a
// caller may choose to have it in the type of x, half the bytes of the last two steps
// (4096 tokens of 8 choices, 4096 -> 2048 -> 4096 in bf16: 454 us, 536 in fp32).
int ffn_y_dtype(const nvfp4_moe_options_t& opt, int dtype) {
  return opt.round_outputs ? dtype : NVFP4_DTYPE_FP32;
}

// Byte offsets of moe_ffn's workspace.
struct FfnSpace {
  int64_t rows, counts, starts, plan, xq, xsf, hq, hsf, y, bytes;
};

FfnSpace ffn_space(const MoeShape& s, int64_t E, int64_t D, int64_t F) {
  FfnSpace w;
  int64_t at = 0;
  auto take = [&at](int64_t bytes) {
    const int64_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  w.rows = take(s.choices * 4);
  w.counts = take(E * 4);
  w.starts = take(E * 4);
  w.plan = take(s.bytes);
  w.xq = take(s.rows * (D / 2));
  w.xsf = take(s.rows / 128 * ceil_div(D, 64) * 512);
  w.hq = take(s.rows * (F / 2));
  w.hsf = take(s.rows / 128 * ceil_div(F, 64) * 512);
  w.y = take(s.tiles * s.tile_rows * D * 4);  // (compact tiles)
  w.bytes = at;
  return w;
}

// compact: c's tiles follow each other, whatever their rows.
nvfp4_status_t moe_product(const void* a, const void* sfa, const void* b, const void* sfb, const void* plan, int64_t T,
                           int64_t top_k, int64_t E, int64_t M, int64_t K, const float* alpha, int activation, void* c,
                           int c_dtype, bool compact, CUstream_st* stream) {
  nvfp4_status_t st = validate_moe(T, top_k, E);
  if (st != NVFP4_OK) return st;
  const MoeShape s = moe_shape(T, top_k, E);
  st = validate_grouped(s, M, K, E);
  if (st != NVFP4_OK) return st;
  if (!valid_dtype(c_dtype) || !valid_activation(activation)) return NVFP4_ERR_INVALID_VALUE;
  if (K == 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (T == 0 || M == 0) return NVFP4_OK;
  if (a == nullptr || sfa == nullptr || b == nullptr || sfb == nullptr || plan == nullptr || c == nullptr)
    return NVFP4_ERR_INVALID_VALUE;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(sfa, 16) || !aligned(sfb, 16) || !aligned(plan, 16) ||
      !aligned(alpha, 4) || !aligned(c, dtype_size(c_dtype)))
    return NVFP4_ERR_MISALIGNED;
  int sms = 0;
  const cudaError_t err = sm_count(&sms);
  if (err != cudaSuccess) return result(err);
  GemmArgs g = moe_gemm_args(a, sfa, b, sfb, plan, s, E, M, K);
  g.alphas = alpha;
  g.activation = activation;
  g.c = c;
  g.c_dtype = c_dtype;
  g.c_stride = M;
  g.compact = compact;
  return result(launch_gemm(g, sms, (cudaStream_t)stream));
}

// skip: see CombineParams.
nvfp4_status_t combine(const void* y, int y_dtype, const int32_t* rows, const float* weights, int64_t T, int64_t top_k,
                       int64_t M, void* out, int dtype, int skip, CUstream_st* stream) {
  if ((dtype != NVFP4_DTYPE_FP16 && dtype != NVFP4_DTYPE_BF16) ||
      (y_dtype != dtype && y_dtype != NVFP4_DTYPE_FP32) || T < 0 || top_k < 1 || M < 0)
    return NVFP4_ERR_INVALID_VALUE;
  if (M % 8 != 0 || M > kMaxK || top_k > kMaxTopK || T > kMaxChoices) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (T == 0 || M == 0) return NVFP4_OK;
  if (y == nullptr || rows == nullptr || weights == nullptr || out == nullptr) return NVFP4_ERR_INVALID_VALUE;
  if (!aligned(y, 16) || !aligned(rows, 4) || !aligned(weights, 4) || !aligned(out, 16))
    return NVFP4_ERR_MISALIGNED;
  int sms = 0;
  const cudaError_t err = sm_count(&sms);
  if (err != cudaSuccess) return result(err);
  CombineParams p = {};
  p.y = y;
  p.rows = rows;
  p.weights = weights;
  p.out = out;
  p.T = T;
  p.M = M;
  p.k = (int32_t)top_k;
  p.skip = skip;
  return result(launch_combine(p, y_dtype, dtype, sms, (cudaStream_t)stream));
}

}  // namespace

extern "C" {

nvfp4_status_t nvfp4_quantize(const void* x, int x_dtype, int64_t x_row_stride, int64_t rows, int64_t K,
                              int64_t L, float encode_scale, void* q, void* sf, int sf_layout,
                              const int32_t* row_map, int copies, int64_t q_rows,
                              struct CUstream_st* stream) {
  nvfp4_status_t st = validate_rows(x_dtype, rows, K, L, x_row_stride, sf_layout);
  if (st != NVFP4_OK) return st;
  if (!(encode_scale > 0.f) || !std::isfinite(encode_scale)) return NVFP4_ERR_INVALID_VALUE;
  if (row_map != nullptr && (copies < 1 || q_rows < 0 || L > 1)) return NVFP4_ERR_INVALID_VALUE;
  if (row_map != nullptr && (copies > kMaxTopK || q_rows > kMaxDim)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0 || K == 0 || L == 0) return NVFP4_OK;
  if (x == nullptr || q == nullptr || sf == nullptr) return NVFP4_ERR_INVALID_VALUE;
  if (!aligned(x, dtype_size(x_dtype)) || !aligned(q, 8) || !aligned(sf, 4) || !aligned(row_map, 4))
    return NVFP4_ERR_MISALIGNED;
  int sms = 0;
  const cudaError_t err = sm_count(&sms);
  if (err != cudaSuccess) return result(err);
  QuantizeParams p = {};
  p.x = x;
  p.q = static_cast<uint8_t*>(q);
  p.sf = static_cast<uint8_t*>(sf);
  p.row_map = row_map;
  p.q_rows = q_rows;
  p.rows = rows;
  p.x_stride = x_row_stride ? x_row_stride : K;
  p.encode = encode_scale;
  p.copies = copies;
  p.half_k = (int32_t)(K / 2);
  p.blocks = (int32_t)(K / 16);
  p.rest_k = (int32_t)ceil_div(K, 64);
  return result(launch_quantize(p, x_dtype, sf_layout == NVFP4_SF_PERMUTED_128x4, L, sms,
                                (cudaStream_t)stream));
}

nvfp4_status_t nvfp4_dequantize(const void* q, const void* sf, int sf_layout, int64_t rows, int64_t K,
                                int64_t L, float scale, void* x, int x_dtype, int64_t x_row_stride,
                                struct CUstream_st* stream) {
  nvfp4_status_t st = validate_rows(x_dtype, rows, K, L, x_row_stride, sf_layout);
  if (st != NVFP4_OK) return st;
  if (rows == 0 || K == 0 || L == 0) return NVFP4_OK;
  if (x == nullptr || q == nullptr || sf == nullptr) return NVFP4_ERR_INVALID_VALUE;
  if (!aligned(x, dtype_size(x_dtype)) || !aligned(q, 8)) return NVFP4_ERR_MISALIGNED;
  int sms = 0;
  const cudaError_t err = sm_count(&sms);
  if (err != cudaSuccess) return result(err);
  DequantizeParams p = {};
  p.q = static_cast<const uint8_t*>(q);
  p.sf = static_cast<const uint8_t*>(sf);
  p.x = x;
  p.rows = rows;
  p.L = L;
  p.x_stride = x_row_stride ? x_row_stride : K;
  p.scale = scale;
  p.half_k = (int32_t)(K / 2);
  p.blocks = (int32_t)(K / 16);
  p.rest_k = (int32_t)ceil_div(K, 64);
  p.permuted = sf_layout == NVFP4_SF_PERMUTED_128x4;
  return result(launch_dequantize(p, x_dtype, sms, (cudaStream_t)stream));
}

nvfp4_status_t nvfp4_fold_scale_signs(void* a, void* sf, int sf_layout, int64_t rows, int64_t K, int64_t L,
                                      struct CUstream_st* stream) {
  nvfp4_status_t st = validate_rows(NVFP4_DTYPE_FP16, rows, K, L, 0, sf_layout);
  if (st != NVFP4_OK) return st;
  if (rows == 0 || K == 0 || L == 0) return NVFP4_OK;
  if (a == nullptr || sf == nullptr) return NVFP4_ERR_INVALID_VALUE;
  if (!aligned(a, 8)) return NVFP4_ERR_MISALIGNED;
  int sms = 0;
  const cudaError_t err = sm_count(&sms);
  if (err != cudaSuccess) return result(err);
  FoldParams p = {};
  p.a = static_cast<uint8_t*>(a);
  p.sf = static_cast<uint8_t*>(sf);
  p.rows = rows;
  p.L = L;
  p.half_k = (int32_t)(K / 2);
  p.blocks = (int32_t)(K / 16);
  p.rest_k = (int32_t)ceil_div(K, 64);
  p.permuted = sf_layout == NVFP4_SF_PERMUTED_128x4;
  return result(launch_fold_signs(p, sms, (cudaStream_t)stream));
}

nvfp4_status_t nvfp4_gemm(const void* a, const void* b, const void* sfa, const void* sfb, void* c,
                          int64_t M, int64_t N, int64_t K, int64_t L,
                          const nvfp4_gemm_options_t* options, struct CUstream_st* stream) {
  static const nvfp4_gemm_options_t kDefaults = {1.0f, nullptr, NVFP4_ACT_NONE, NVFP4_DTYPE_FP16, 0};
  const nvfp4_gemm_options_t& opt = options ? *options : kDefaults;
  nvfp4_status_t st = validate_product(M, N, K, L);
  if (st != NVFP4_OK) return st;
  if (!dense_tiles_fit(M, N, L)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!valid_dtype(opt.c_dtype) || !valid_activation(opt.activation) ||
      (opt.c_row_stride != 0 && opt.c_row_stride < M))
    return NVFP4_ERR_INVALID_VALUE;
  if (M == 0 || N == 0 || L == 0) return NVFP4_OK;
  if (c == nullptr || (K != 0 && (a == nullptr || b == nullptr || sfa == nullptr || sfb == nullptr)))
    return NVFP4_ERR_INVALID_VALUE;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(sfa, 16) || !aligned(sfb, 16) ||
      !aligned(c, dtype_size(opt.c_dtype)) || !aligned(opt.bias, 4))
    return NVFP4_ERR_MISALIGNED;
  int sms = 0;
  const cudaError_t err = sm_count(&sms);
  if (err != cudaSuccess) return result(err);
  GemmArgs g = {};
  g.a = static_cast<const uint8_t*>(a);
  g.sfa = static_cast<const uint8_t*>(sfa);
  g.b = static_cast<const uint8_t*>(b);
  g.sfb = static_cast<const uint8_t*>(sfb);
  g.M = M;
  g.N = N;
  g.K = K;
  g.G = L;
  g.c = c;
  g.c_dtype = opt.c_dtype;
  g.c_stride = opt.c_row_stride ? opt.c_row_stride : M;
  g.bias = opt.bias;
  g.alpha = opt.alpha;
  g.activation = opt.activation;
  return result(launch_gemm(g, sms, (cudaStream_t)stream));
}

nvfp4_status_t nvfp4_gemm_plan(int64_t M, int64_t N, int64_t K, int64_t L, int num_sms, int* tile_rows,
                               int* k_split) {
  if (tile_rows == nullptr || k_split == nullptr || num_sms < 2) return NVFP4_ERR_INVALID_VALUE;
  const nvfp4_status_t st = validate_product(M, N, K, L);
  if (st != NVFP4_OK) return st;
  if (!dense_tiles_fit(M, N, L)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  const GemmChoice c = choose_gemm(M < 1 ? 1 : M, N < 1 ? 1 : N, K < 1 ? 1 : K, L < 1 ? 1 : L, num_sms, false);
  *tile_rows = c.bn;
  *k_split = c.ks;
  return NVFP4_OK;
}

nvfp4_status_t nvfp4_route(const void* logits, int dtype, int64_t row_stride, int64_t T, int64_t E,
                           int top_k, const nvfp4_route_options_t* options, int32_t* ids, float* weights,
                           struct CUstream_st* stream) {
  static const nvfp4_route_options_t kDefaults = {NVFP4_SCORE_SOFTMAX, nullptr, 1, 1, 1, 1.0f};
  const nvfp4_route_options_t& opt = options ? *options : kDefaults;
  if (!valid_dtype(dtype) || T < 0 || E < 1 || top_k < 1 || (row_stride != 0 && row_stride < E))
    return NVFP4_ERR_INVALID_VALUE;
  if ((opt.score != NVFP4_SCORE_SOFTMAX && opt.score != NVFP4_SCORE_SIGMOID) || opt.groups < 1 ||
      opt.top_groups < 1 || opt.top_groups > opt.groups)
    return NVFP4_ERR_INVALID_VALUE;
  if (E > kMaxExperts || top_k > kMaxTopK || top_k > E || opt.groups > kMaxGroups || E % opt.groups != 0 ||
      T > kMaxRows)
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return NVFP4_OK;
  if (logits == nullptr || ids == nullptr || weights == nullptr) return NVFP4_ERR_INVALID_VALUE;
  if (!aligned(logits, dtype_size(dtype)) || !aligned(opt.bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
    return NVFP4_ERR_MISALIGNED;
  int sms = 0;
  const cudaError_t err = sm_count(&sms);
  if (err != cudaSuccess) return result(err);
  RouteParams p = {};
  p.logits = logits;
  p.bias = opt.bias;
  p.ids = ids;
  p.weights = weights;
  p.T = T;
  p.stride = row_stride ? row_stride : E;
  p.scale = opt.weight_scale;
  p.E = (int32_t)E;
  p.k = top_k;
  p.groups = opt.groups;
  p.top_groups = opt.top_groups;
  p.sigmoid = opt.score == NVFP4_SCORE_SIGMOID;
  p.renormalize = opt.renormalize;
  return result(launch_route(p, dtype, sms, (cudaStream_t)stream));
}

nvfp4_status_t nvfp4_moe_shape(int64_t T, int64_t top_k, int64_t E, nvfp4_moe_shape_t* out) {
  if (out == nullptr) return NVFP4_ERR_INVALID_VALUE;
  const nvfp4_status_t st = validate_moe(T, top_k, E);
  if (st != NVFP4_OK) return st;
  const MoeShape s = moe_shape(T, top_k, E);
  out->tile_rows = s.tile_rows;
  out->row_capacity = s.rows;
  out->plan_bytes = (size_t)s.bytes;
  return NVFP4_OK;
}

nvfp4_status_t nvfp4_moe_sort(const int32_t* ids, int64_t T, int64_t top_k, int64_t E, int32_t* rows,
                              int32_t* counts, int32_t* starts, void* plan, struct CUstream_st* stream) {
  const nvfp4_status_t st = validate_moe(T, top_k, E);
  if (st != NVFP4_OK) return st;
  if ((T != 0 && (ids == nullptr || rows == nullptr)) || counts == nullptr || starts == nullptr ||
      plan == nullptr)
    return NVFP4_ERR_INVALID_VALUE;
  if (!aligned(ids, 4) || !aligned(rows, 4) || !aligned(counts, 4) || !aligned(starts, 4) ||
      !aligned(plan, 16))
    return NVFP4_ERR_MISALIGNED;
  return result(launch_sort(sort_params(ids, moe_shape(T, top_k, E), E, rows, counts, starts, plan),
                            (cudaStream_t)stream));
}

nvfp4_status_t nvfp4_moe_gemm(const void* a, const void* sfa, const void* b, const void* sfb,
                              const void* plan, int64_t T, int64_t top_k, int64_t E, int64_t M, int64_t K,
                              const float* alpha, int activation, void* c, int c_dtype,
                              struct CUstream_st* stream) {
  return moe_product(a, sfa, b, sfb, plan, T, top_k, E, M, K, alpha, activation, c, c_dtype, false, stream);
}

nvfp4_status_t nvfp4_moe_gated_gemm(const void* a, const void* sfa, const void* b, const void* sfb,
                                    const void* plan, int64_t T, int64_t top_k, int64_t E, int64_t F,
                                    int64_t K, const float* alpha, int activation, float encode_scale,
                                    void* q, void* sf, struct CUstream_st* stream) {
  nvfp4_status_t st = validate_moe(T, top_k, E);
  if (st != NVFP4_OK) return st;
  if (F < 0 || F > kMaxDim / 2) return NVFP4_ERR_INVALID_VALUE;
  const MoeShape s = moe_shape(T, top_k, E);
  st = validate_grouped(s, 2 * F, K, E);
  if (st != NVFP4_OK) return st;
  if (!valid_activation(activation) || !(encode_scale > 0.f) || !std::isfinite(encode_scale))
    return NVFP4_ERR_INVALID_VALUE;
  if (K == 0 || F % 32 != 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (T == 0 || F == 0) return NVFP4_OK;
  if (a == nullptr || sfa == nullptr || b == nullptr || sfb == nullptr || plan == nullptr || q == nullptr ||
      sf == nullptr)
    return NVFP4_ERR_INVALID_VALUE;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(sfa, 16) || !aligned(sfb, 16) || !aligned(plan, 16) ||
      !aligned(alpha, 4) || !aligned(q, 16) || !aligned(sf, 16))
    return NVFP4_ERR_MISALIGNED;
  int sms = 0;
  const cudaError_t err = sm_count(&sms);
  if (err != cudaSuccess) return result(err);
  GemmArgs g = moe_gemm_args(a, sfa, b, sfb, plan, s, E, 2 * F, K);
  g.alphas = alpha;
  g.activation = activation;
  g.q = static_cast<uint8_t*>(q);
  g.qsf = static_cast<uint8_t*>(sf);
  g.encode = encode_scale;
  return result(launch_gemm(g, sms, (cudaStream_t)stream));
}

nvfp4_status_t nvfp4_moe_combine(const void* y, int y_dtype, const int32_t* rows, const float* weights,
                                 int64_t T, int64_t top_k, int64_t M, void* out, int dtype,
                                 struct CUstream_st* stream) {
  return combine(y, y_dtype, rows, weights, T, top_k, M, out, dtype, 0, stream);
}

size_t nvfp4_moe_ffn_workspace_bytes(int64_t T, int64_t top_k, int64_t E, int64_t D, int64_t F) {
  if (validate_ffn(T, top_k, E, D, F) != NVFP4_OK) return 0;
  return (size_t)ffn_space(moe_shape(T, top_k, E), E, D, F).bytes;
}

nvfp4_status_t nvfp4_moe_ffn(const void* x, int dtype, int64_t x_row_stride, const int32_t* ids,
                             const float* weights, const void* w1, const void* sf1, const void* w2,
                             const void* sf2, int64_t T, int64_t top_k, int64_t E, int64_t D, int64_t F,
                             const nvfp4_moe_options_t* options, void* out, void* workspace,
                             size_t workspace_bytes, struct CUstream_st* stream) {
  static const nvfp4_moe_options_t kDefaults = {nullptr, nullptr, 1.0f, 1.0f, NVFP4_ACT_SILU, 0};
  const nvfp4_moe_options_t& opt = options ? *options : kDefaults;
  nvfp4_status_t st = validate_moe(T, top_k, E);
  if (st != NVFP4_OK) return st;
  if ((dtype != NVFP4_DTYPE_FP16 && dtype != NVFP4_DTYPE_BF16) || D < 0 || F < 0 ||
      (x_row_stride != 0 && x_row_stride < D) || !valid_activation(opt.activation) ||
      !(opt.encode_x > 0.f) || !std::isfinite(opt.encode_x) || !(opt.encode_h > 0.f) ||
      !std::isfinite(opt.encode_h) || (opt.round_outputs != 0 && opt.round_outputs != 1))
    return NVFP4_ERR_INVALID_VALUE;
  if ((st = validate_ffn(T, top_k, E, D, F)) != NVFP4_OK ||
      (st = validate_rows(dtype, T, D, 1, x_row_stride, NVFP4_SF_PERMUTED_128x4)) != NVFP4_OK)
    return st;
  const MoeShape s = moe_shape(T, top_k, E);
  if (T == 0) return NVFP4_OK;
  const FfnSpace w = ffn_space(s, E, D, F);
  if (x == nullptr || ids == nullptr || weights == nullptr || w1 == nullptr || sf1 == nullptr ||
      w2 == nullptr || sf2 == nullptr || out == nullptr || workspace == nullptr ||
      workspace_bytes < (size_t)w.bytes)
    return NVFP4_ERR_INVALID_VALUE;
  if (!aligned(x, 2) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(w1, 16) || !aligned(sf1, 16) ||
      !aligned(w2, 16) || !aligned(sf2, 16) || !aligned(out, 16) || !aligned(workspace, 256) ||
      !aligned(opt.alpha1, 4) || !aligned(opt.alpha2, 4))
    return NVFP4_ERR_MISALIGNED;
  uint8_t* const base = static_cast<uint8_t*>(workspace);
  int32_t* const rows = reinterpret_cast<int32_t*>(base + w.rows);
  int32_t* const counts = reinterpret_cast<int32_t*>(base + w.counts);
  int32_t* const starts = reinterpret_cast<int32_t*>(base + w.starts);
  int skip = s.pitch > 128 ? 0 : 128 - s.tile_rows;  // (the outputs' tiles follow each other)
  if (s.choices <= kPlaceMost) {
    PlaceParams p = {};
    p.skip = skip;
    skip = 0;
    p.sort = sort_params(ids, s, E, rows, counts, starts, base + w.plan);
    p.quantize.x = x;
    p.quantize.q = base + w.xq;
    p.quantize.sf = base + w.xsf;
    p.quantize.x_stride = x_row_stride ? x_row_stride : D;
    p.quantize.encode = opt.encode_x;
    p.quantize.copies = (int32_t)top_k;
    p.quantize.half_k = (int32_t)(D / 2);
    p.quantize.blocks = (int32_t)(D / 16);
    p.quantize.rest_k = (int32_t)ceil_div(D, 64);
    st = result(launch_place(p, dtype, T, (cudaStream_t)stream));
    if (st != NVFP4_OK) return st;
  } else {
    st = nvfp4_moe_sort(ids, T, top_k, E, rows, counts, starts, base + w.plan, stream);
    if (st != NVFP4_OK) return st;
    st = nvfp4_quantize(x, dtype, x_row_stride, T, D, 1, opt.encode_x, base + w.xq, base + w.xsf,
                        NVFP4_SF_PERMUTED_128x4, rows, (int)top_k, s.rows, stream);
    if (st != NVFP4_OK) return st;
  }
  st = nvfp4_moe_gated_gemm(w1, sf1, base + w.xq, base + w.xsf, base + w.plan, T, top_k, E, F, D, opt.alpha1,
                            opt.activation, opt.encode_h, base + w.hq, base + w.hsf, stream);
  if (st != NVFP4_OK) return st;
  const int y_dtype = ffn_y_dtype(opt, dtype);
  st = moe_product(w2, sf2, base + w.hq, base + w.hsf, base + w.plan, T, top_k, E, D, F, opt.alpha2, NVFP4_ACT_NONE,
                   base + w.y, y_dtype, true, stream);
  if (st != NVFP4_OK) return st;
  return combine(base + w.y, y_dtype, rows, weights, T, top_k, D, out, dtype, skip, stream);
}

}  // extern "C"
