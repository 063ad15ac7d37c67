// Host/device interface of the layer operators: quantise, the product for any
// number of rows, routing, and the routed experts.
#pragma once
#include <atomic>
#include <cstdint>

#include <cuda_runtime.h>

namespace nvfp4 {

enum DataType { kF16 = 0, kBF16 = 1, kF32 = 2 };  // nvfp4_dtype_t

// Remembers a failed runtime call for nvfp4_last_cuda_error and clears a
// non-sticky launch error (api.cu).
void record_cuda_error(cudaError_t err);

// Launch with programmatic stream serialization (the kernel waits for the
// preceding work itself, with pdl_wait, before it touches memory).
template <typename P>
inline cudaError_t launch_pdl(void (*kern)(P), dim3 grid, dim3 block, size_t smem,
                              cudaStream_t stream, const P& p, int cluster = 1) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

// Allows the kernel its dynamic shared memory, once per device (each kernel
// asks for one size only).
template <auto KERN>
inline cudaError_t allow_smem(size_t bytes) {
  static std::atomic<uint64_t> done[2];  // a bit per device (of the first 128)
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (done[dev >> 6].load(std::memory_order_relaxed) & bit) return cudaSuccess;
  err = cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (err == cudaSuccess) done[dev >> 6].fetch_or(bit, std::memory_order_relaxed);
  return err;
}

// ---- quantise / dequantise (quantize.cu) ----

struct QuantizeParams {
  const void* x;      // [L][rows] rows of x_stride elements
  uint8_t* q;         // [L][rows][K/2], or with row_map [q_rows][K/2]
  uint8_t* sf;        // scales of those rows
  const int32_t* row_map;  // [rows][copies]: rows of q that a row of x goes to, or null
  int64_t q_rows;     // rows of q with a row_map (entries outside [0, q_rows) are skipped)
  int64_t rows, rows_pad, x_stride;
  int64_t places;     // set by the launcher
  float encode;
  int32_t copies, half_k, blocks, rest_k, one_batch, chunks;
};
cudaError_t launch_quantize(QuantizeParams p, int dtype, bool permuted, int64_t L, int sms,
                            cudaStream_t stream);

struct DequantizeParams {
  const uint8_t* q;
  const uint8_t* sf;
  void* x;
  int64_t rows, L, x_stride;
  int64_t places;     // set by the launcher
  float scale;
  int32_t half_k, blocks, rest_k, chunks;
  bool permuted;
};
cudaError_t launch_dequantize(DequantizeParams p, int dtype, int sms, cudaStream_t stream);

struct FoldParams {
  uint8_t* a;
  uint8_t* sf;
  int64_t rows, L;
  int32_t half_k, blocks, rest_k;
  bool permuted;
};
cudaError_t launch_fold_signs(const FoldParams& p, int sms, cudaStream_t stream);

// ---- the product (gemm_tc.cu) ----

// Dense (groups = batches) or grouped (groups = experts, token tiles from a
// device table).
struct GemmArgs {
  const uint8_t* a;    // [G][M][K/2]
  const uint8_t* sfa;  // 128x4 atoms per group
  const uint8_t* b;    // dense [L][N][K/2]; grouped [rows][K/2]
  const uint8_t* sfb;  // 128x4 atoms (grouped: of all rows)
  int64_t M, N, K, G;  // N: rows of b per batch; grouped: all rows of b
  // grouped: tiles of token rows {expert, first row, rows, 0} and their number, on the device
  const int4* tiles;
  const int32_t* tile_count;
  int64_t max_tiles;   // upper bound of *tile_count
  int tile_rows;       // rows of a grouped tile (the kernel's N tile)
  bool compact;        // c's tiles of fewer than 128 rows follow each other (see CombineParams)
  // epilogue
  void* c;             // [G or 1][N][c_stride], or null with a quantised output
  int c_dtype;
  int64_t c_stride;
  const float* bias;   // [G][M] or null
  const float* alphas; // [G] or null
  float alpha;
  int activation;
  // quantised gated output: rows of K = M/2
  uint8_t* q;
  uint8_t* qsf;
  float encode;
};
cudaError_t launch_gemm(const GemmArgs& g, int sms, cudaStream_t stream);
cudaError_t gemm_wait_timeouts(int reset, int* out);
// What a product's CTA takes of its SM (see gemm::most_columns).
struct Footprint {
  uint32_t smem, columns;  // dynamic shared memory; tensor memory
};
Footprint product_footprint(int tile_rows, bool gated);
// The dense product's rows of b per tile and CTAs that split a tile's K.
struct GemmChoice {
  int bn, ks;
};
GemmChoice choose_gemm(int64_t M, int64_t N, int64_t K, int64_t L, int sms, bool activation);

// ---- routing and the experts' rows (route.cu, moe.cu) ----

struct RouteParams {
  const void* logits;  // [T] rows of stride elements
  const float* bias;   // [E] or null
  int32_t* ids;        // [T][k]
  float* weights;      // [T][k]
  int64_t T, stride;
  float scale;
  int32_t E, k, groups, top_groups, sigmoid, renormalize;
  // set by the launcher: the rows' alignment (up to 16), a group's experts, and the lanes
  // that hold them as a power of two (-1: they do not fill lanes of their own)
  int32_t aligned, per_group, lanes_log2;
};
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;
constexpr int kMaxGroups = 32;
cudaError_t launch_route(RouteParams p, int dtype, int sms, cudaStream_t stream);

// Where the sort leaves its results: counts [E], tiles and their number, and
// each choice's row.
struct SortParams {
  const int32_t* ids;  // [T*k]; outside [0, E): no expert
  int32_t* rows;       // [T*k]: row of the choice, or -1
  int32_t* counts;     // [E]
  int32_t* starts;     // [E]: first row
  int4* tiles;
  int32_t* tile_count;
  int32_t* chunk_counts;  // [chunks][E] scratch
  int64_t n;           // T*k
  int32_t E, tile_rows, pitch;  // a tile's rows, and rows from one tile to the next
};
constexpr int kSortThreads = 512;
constexpr int kSortChunk = 4096;  // choices per CTA
cudaError_t launch_sort(const SortParams& p, cudaStream_t stream);

// The sort and the quantisation into the experts' rows of few choices in one launch
// (quantize.cu): sort.n = T * quantize.copies <= kPlaceMost, 16-bit x.
constexpr int kPlaceMost = 1024;
struct PlaceParams {
  SortParams sort;
  QuantizeParams quantize;
  int32_t skip;  // sort.rows is written for CombineParams with these already left out
};
cudaError_t launch_place(const PlaceParams& p, int dtype, int64_t T, cudaStream_t stream);

struct CombineParams {
  const void* y;       // [rows][M], fp32 or the type of out
  const int32_t* rows; // [T][k]
  const float* weights;
  void* out;           // [T][M]
  int64_t T, M;
  int32_t k;
  // rows that y leaves out of each 128 that `rows` counts: 0, or, if y's tiles of fewer rows
  // follow each other, 128 less a tile's (a scale atom's rows mean nothing to y, and are 8 times
  // the memory of tiles of 16)
  int32_t skip;
};
cudaError_t launch_combine(const CombineParams& p, int y_dtype, int dtype, int sms, cudaStream_t stream);

}  // namespace nvfp4
