// NVFP4 product for any number of rows, on the tensor cores (tcgen05, sm_103a):
//   c[n][m] = act(alpha * sum_k A[m][k] * B[n][k] + bias[m])
// with A (the weights) and B (the tokens) E2M1 with one E4M3 scale per 16
// elements, scales in 128x4 atoms.  Dense (one B per batch) or grouped: every
// token tile names the expert whose A it multiplies, from a table that the
// sort of the routed choices leaves on the device.
//
// The block-scaled MMA (kind::mxf4nvf4, 16-element blocks) takes 128 rows of A
// and BN rows of B per instruction, K = 64, and accumulates in fp32 in tensor
// memory; weights are the M operand, so a few tokens cost a narrow N tile and
// not a padded 128-row one.  A stage is 256 elements of K: a 128-byte row of
// either operand (TMA, 128-byte swizzle) and four scale atoms of 512 bytes per
// 128 rows, adjacent in memory (bulk copies).  The atoms are copied to tensor
// memory as they are (tcgen05.cp), into columns that belong to the stage, so
// nothing there is overwritten before the stage's MMAs have been committed.
//
// One CTA (192 threads) per SM, persistent over the tiles:
//   warp 0     one lane issues the copies of every stage
//   warp 1     allocates tensor memory; one lane issues TMEM copies and MMAs
//   warps 2-5  read the accumulator (a TMEM lane quarter each) and store c, or
//              quantise the gated activation
// Tiles of 256 rows of B run on pairs of SMs instead (gemm_pair.cu).
//
// What bounds it: with few rows per expert the weights' bytes (53 tokens through 8 of 64
// experts, 4096 -> 2048 -> 4096: 107 to 125 us for the layer, the weights of the 39 to 49
// experts in use at the measured copy rate); for one small matrix the latency of a CTA's stages, one
// after another, which is why idle SMs split a tile's K (1 x 4096 x 4096: 5.6 us, 7.0 without);
// with 128 rows the bytes of a stage into shared memory, 36 KB at ~64 bytes per cycle and SM.
//
// Scale codes are unsigned magnitudes (the MMA ignores bit 7).
//
// Every wait on an mbarrier gives up after tc::kWaitNs, counts a timeout in a
// device word the host can read, and the thread then skips its remaining work.
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>

#include "attention.h"
#include "gemm_common.cuh"

namespace nvfp4 {

__device__ int g_gemm_timeouts;

namespace {

using namespace gemm;

constexpr int kGemmThreads = 192;

__host__ __device__ constexpr uint32_t stage_bytes(int bn) { return kABytes + (uint32_t)bn * 128u + 2 * kAtoms; }
__host__ __device__ constexpr int stages_for(int bn) { return bn == 128 ? 5 : 6; }
constexpr int kAcc = 2;  // accumulators in tensor memory
// Accumulators, then 16 columns of either operand's scales per stage (allocated as a power of two).
__host__ __device__ constexpr uint32_t columns_for(int bn) {
  return (uint32_t)(kAcc * bn + 32 * stages_for(bn)) <= 256u ? 256u : 512u;
}
constexpr uint32_t gemm_smem_bytes(int bn, int epi) {
  const uint32_t bytes = (uint32_t)stages_for(bn) * stage_bytes(bn) + 1024u +
                         (epi == kGatedQuantize ? 4u * kTransposeBytes : 0u);
  return columns_for(bn) == 512 && bytes < kAloneSmem ? kAloneSmem : bytes;
}
constexpr bool columns_fit(int bn) {
  return most_columns(gemm_smem_bytes(bn, kStore), columns_for(bn)) <= 512 &&
         most_columns(gemm_smem_bytes(bn, kGatedQuantize), columns_for(bn)) <= 512;
}
static_assert(columns_fit(16) && columns_fit(32) && columns_fit(64) && columns_fit(128), "tensor memory of an SM");

template <typename T>
__device__ __forceinline__ void store_one(const GemmParams& p, int64_t idx, float v) {
  static_cast<T*>(p.c)[idx] = round_to(T(), v);
}

// NC floats at p of the CTA of the given cluster rank, added to v.
__device__ __forceinline__ void add_remote(uint32_t saddr, uint32_t rank, float (&v)[kUnit]) {
  const uint32_t at = tc::map_rank(saddr, rank);
#pragma unroll
  for (int i = 0; i < kUnit; ++i) {
    float f;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(at + 512u * i) : "memory");
    v[i] += f;
  }
}

// SPLIT: the CTAs of a cluster take one tile, a part of its K stages each; the
// others leave their sums in their own shared memory (the ring's, no longer in use)
// and rank 0 adds them in rank order.
template <int BN, int EPI, bool GROUPED, bool SPLIT>
__global__ void __launch_bounds__(kGemmThreads, 1) gemm_kernel(const __grid_constant__ GemmParams p) {
  constexpr int S = stages_for(BN);
  constexpr uint32_t kSfaCol = kAcc * BN;
  constexpr uint32_t kSfbCol = kSfaCol + 16 * S;
  constexpr uint32_t kColumns = columns_for(BN);
  static_assert(kSfbCol + 16 * S <= kColumns, "TMEM columns");
  extern __shared__ uint8_t gemm_smem[];
  __shared__ __align__(8) uint64_t bars[2 * S + 2 * kAcc + 1];
  __shared__ uint32_t tmem_slot;

  const uint32_t raw = smem_u32(gemm_smem);
  const uint32_t a_s = (raw + 1023u) & ~1023u;
  const uint32_t b_s = a_s + S * kABytes;
  const uint32_t sfa_s = b_s + S * BN * 128u;
  const uint32_t sfb_s = sfa_s + S * kAtoms;
  const uint32_t tr_s = sfb_s + S * kAtoms;
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int st) { return bar0 + 8u * st; };
  auto empty_bar = [&](int st) { return bar0 + 8u * (S + st); };
  auto dfull_bar = [&](int i) { return bar0 + 8u * (2 * S + i); };
  auto dempty_bar = [&](int i) { return bar0 + 8u * (2 * S + kAcc + i); };
  const uint32_t drain_bar = bar0 + 8u * (2 * S + 2 * kAcc);

  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int st = 0; st < S; ++st) {
      tc::mbar_init(full_bar(st), 1);
      tc::mbar_init(empty_bar(st), 1);
    }
    for (int i = 0; i < kAcc; ++i) {
      tc::mbar_init(dfull_bar(i), 1);
      tc::mbar_init(dempty_bar(i), 4);
    }
    tc::mbar_init(drain_bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // the preceding kernels have ended before tensor memory is taken (a kernel
  // that this one waits for may not have taken its own yet), and the next one
  // may start only after that
  pdl_wait();
  if (warp == 1) tc::alloc(smem_u32(&tmem_slot), kColumns);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
  const int32_t total = GROUPED ? __shfl_sync(0xffffffffu, *p.tile_count, 0) * p.tiles_m : p.total;
  bool ok = true;
  const int ks = SPLIT ? (int)tc::cluster_size() : 1, rank = SPLIT ? (int)tc::cluster_rank() : 0;
  const int32_t first = (int32_t)blockIdx.x / ks, step = (int32_t)gridDim.x / ks;
  // this CTA's stages of a tile (with SPLIT every rank has some)
  const int s_begin = SPLIT ? p.kstages * rank / ks : 0;
  const int s_end = SPLIT ? p.kstages * (rank + 1) / ks : p.kstages;
  static_assert(!SPLIT || (uint32_t)BN * 128 * 4 <= S * kABytes, "the sums fit the ring");

  if (warp == 0) {
    int pos = 0, issued = 0;
    uint32_t ph = 0;
    for (int32_t t = first; t < total; t += step) {
      const Tile tile = tile_at<BN, GROUPED>(p, t);
      const int64_t batch = GROUPED ? 0 : tile.g;
      const uint8_t* sa = p.sfa + ((int64_t)tile.g * p.rest_m + tile.mt) * p.rest_k * 512;
      const uint8_t* sb = p.sfb + (batch * p.rest_n + tile.n0 / 128) * p.rest_k * 512;
      for (int s = s_begin; s < s_end; ++s) {
        const uint32_t nb = (uint32_t)min(4, p.rest_k - 4 * s) * 512u;
        tc::mbar_wait<false>(empty_bar(pos), ph ^ 1u, ok, &g_gemm_timeouts);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
          const uint32_t fb = full_bar(pos);
          if (elect_one()) {
            tc::mbar_expect_tx(fb, kABytes + BN * 128u + 2u * nb);
            tc::tma_load_3d(a_s + pos * kABytes, &p.tmap_a, s * 128, tile.mt * 128, tile.g, fb);
            tc::tma_load_3d(b_s + pos * BN * 128u, &p.tmap_b, s * 128, (int)tile.n0, (int)batch, fb);
            tc::bulk_load(sfa_s + pos * kAtoms, sa + (int64_t)s * kAtoms, nb, fb);
            tc::bulk_load(sfb_s + pos * kAtoms, sb + (int64_t)s * kAtoms, nb, fb);
          }
          __syncwarp();
          ++issued;
        }
        if (++pos == S) {
          pos = 0;
          ph ^= 1u;
        }
      }
    }
    // copies still in flight land before the CTA can exit
    bool drain_ok = true;
    for (int k = 0; k < S && k < issued; ++k) {
      const int i = issued - 1 - k;
      tc::mbar_wait<false>(full_bar(i % S), (uint32_t)((i / S) & 1), drain_ok, &g_gemm_timeouts);
    }
    __syncwarp();
  } else if (warp == 1) {
    constexpr uint32_t idesc = tc::mxf4nvf4_idesc(BN);
    int pos = 0, j = 0;
    uint32_t ph = 0;
    for (int32_t t = first; t < total; t += step, ++j) {
      const int acc = j % kAcc;
      const uint32_t d = tmem + acc * BN;
      tc::mbar_wait<false>(dempty_bar(acc), ((uint32_t)(j / kAcc) & 1u) ^ 1u, ok, &g_gemm_timeouts);
      for (int s = s_begin; s < s_end; ++s) {
        const int nk = min(4, p.rest_k - 4 * s);
        tc::mbar_wait<false>(full_bar(pos), ph, ok, &g_gemm_timeouts);
        ok = __all_sync(0xffffffffu, ok);
        tc::fence_after();
        if (ok) {
          const uint32_t ca = tmem + kSfaCol + 16u * pos, cb = tmem + kSfbCol + 16u * pos;
          const uint64_t da = tc::desc_sw128(a_s + pos * kABytes), db = tc::desc_sw128(b_s + pos * BN * 128u);
          const uint64_t dsa = tc::desc_atom(sfa_s + pos * kAtoms);
          const uint64_t dsb = tc::desc_atom(sfb_s + pos * kAtoms);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              if (kk < nk) {
                // (a descriptor counts addresses in units of 16 bytes)
                tc::copy_atom(ca + 4u * kk, dsa + 32u * kk);
                tc::copy_atom(cb + 4u * kk, dsb + 32u * kk);
              }
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              if (kk < nk)
                tc::mma(d, da + 2u * kk, db + 2u * kk, idesc, ca + 4u * kk, cb + 4u * kk, s > s_begin || kk > 0);
            }
            tc::commit(empty_bar(pos));
          }
          __syncwarp();
        }
        if (++pos == S) {
          pos = 0;
          ph ^= 1u;
        }
      }
      if (ok && elect_one()) tc::commit(dfull_bar(acc));
      __syncwarp();
    }
    // every MMA and TMEM copy has finished before TMEM is released
    if (elect_one()) tc::commit(drain_bar);
    bool drain_ok = true;
    tc::mbar_wait<false>(drain_bar, 0, drain_ok, &g_gemm_timeouts);
    __syncwarp();
  } else {
    const int quarter = warp & 3;
    Place w;
    w.transpose = reinterpret_cast<float*>(gemm_smem + (tr_s - raw)) + (warp - 2) * (int)(kTransposeBytes / 4);
    int j = 0;
    for (int32_t t = first; t < total; t += step, ++j) {
      const int acc = j % kAcc;
      const Tile tile = tile_at<BN, GROUPED>(p, t);
      place_at<EPI, GROUPED>(w, p, tile, tile.mt, quarter);
      if (lane == 0) tc::mbar_wait<false>(dfull_bar(acc), (uint32_t)(j / kAcc) & 1u, ok, &g_gemm_timeouts);
      __syncwarp();
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      tc::fence_after();
      const uint32_t d = acc * BN + ((uint32_t)(32 * quarter) << 16);
      // [column][row] sums of the other ranks
      const uint32_t sums = a_s + 4u * (uint32_t)(32 * quarter + lane);
      if (SPLIT && rank > 0) {
        float* const mine = reinterpret_cast<float*>(gemm_smem + (sums - raw));
        for (int n = 0; ok && n < tile.rows; n += kUnit) {
          float v[kUnit];
          tc::tmem_load_cols<kUnit>(tmem + d + n, v);
#pragma unroll
          for (int i = 0; i < kUnit; ++i) mine[(n + i) * 128] = v[i];
        }
      }
      if constexpr (SPLIT) tc::cluster_sync();  // (one tile per cluster; the other warps meet it below)
      if (rank == 0) {
        constexpr int U = BN < 32 || EPI == kGatedQuantize ? 1 : 2;
        for (int n = 0; ok && n < tile.rows; n += U * kUnit) {
          float v[U][kUnit];
          int at[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            at[u] = n + u * kUnit;
            tmem_load_16(tmem + d + at[u], v[u]);
          }
#pragma unroll
          for (int u = 0; u < U; ++u) tmem_wait(v[u]);
          if constexpr (SPLIT)
#pragma unroll
            for (int u = 0; u < U; ++u)
              for (int r = 1; r < ks && at[u] < tile.rows; ++r) add_remote(sums + 512u * at[u], (uint32_t)r, v[u]);
          finish_columns<EPI, U, false>(p, w, at, v);
        }
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(dempty_bar(acc));
    }
  }

  if constexpr (SPLIT) {
    if (warp < 2) tc::cluster_sync();
    tc::cluster_sync();  // rank 0 has read the others' sums
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after();
    tc::dealloc(tmem, kColumns);
  }
}

// alpha * 0 + bias for K = 0.
__global__ void __launch_bounds__(256) gemm_no_k_kernel(const GemmParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t total = p.rows * p.M;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / p.M, m = i - row * p.M;
    float y = p.bias ? p.bias[row / p.N * p.M + m] : 0.f;
    if (p.activation != 0) y = activate(y, p.activation);
    if (p.c_dtype == kF32)
      store_one<float>(p, row * p.c_stride + m, y);
    else if (p.c_dtype == kBF16)
      store_one<__nv_bfloat16>(p, row * p.c_stride + m, y);
    else
      store_one<__half>(p, row * p.c_stride + m, y);
  }
}

template <int BN, int EPI, bool GROUPED, bool SPLIT = false>
cudaError_t launch_variant(const GemmParams& p, int64_t ctas, int ks, cudaStream_t stream) {
  constexpr auto kern = gemm_kernel<BN, EPI, GROUPED, SPLIT>;
  constexpr uint32_t smem = gemm_smem_bytes(BN, EPI);
  cudaError_t err = allow_smem<kern>(smem);
  if (err != cudaSuccess) return err;
  return launch_pdl(kern, dim3((unsigned)ctas), dim3(kGemmThreads), smem, stream, p, ks);
}

template <int BN, int EPI, bool GROUPED>
cudaError_t launch_bn(const GemmParams& p, int64_t max_tiles, int ks, int sms, cudaStream_t stream) {
  if constexpr (EPI == kStore && !GROUPED)
    if (ks > 1) return launch_variant<BN, EPI, false, true>(p, max_tiles * ks, ks, stream);
  return launch_variant<BN, EPI, GROUPED>(p, max_tiles < sms ? max_tiles : sms, 1, stream);
}

template <int EPI, bool GROUPED>
cudaError_t launch_for(int bn, const GemmParams& p, int64_t max_tiles, int ks, int sms, cudaStream_t stream) {
  switch (bn) {
    case 16: return launch_bn<16, EPI, GROUPED>(p, max_tiles, ks, sms, stream);
    case 32: return launch_bn<32, EPI, GROUPED>(p, max_tiles, ks, sms, stream);
    case 64: return launch_bn<64, EPI, GROUPED>(p, max_tiles, ks, sms, stream);
    case 128: return launch_bn<128, EPI, GROUPED>(p, max_tiles, ks, sms, stream);
    case 256: return launch_gemm_pair(p, EPI, GROUPED, max_tiles, sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

// The assertions on most_columns, on the current device; asked once per device.
cudaError_t columns_fit_here(bool* fit) {
  constexpr int kMaxDevices = 128;
  static std::atomic<int> cached[kMaxDevices];  // 0 unknown, 1 they fit, 2 not
  int dev = 0, smem = 0, reserve = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  int c = cached[dev].load(std::memory_order_relaxed);
  if (c == 0) {
    if ((err = cudaDeviceGetAttribute(&smem, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev)) != cudaSuccess ||
        (err = cudaDeviceGetAttribute(&reserve, cudaDevAttrReservedSharedMemoryPerBlock, dev)) != cudaSuccess)
      return err;
    c = 1;
    for (int rows = 16; rows <= 256; rows *= 2)
      for (const bool gated : {false, true}) {
        const Footprint f = product_footprint(rows, gated);
        if (most_columns(f.smem, f.columns, (uint32_t)smem, (uint32_t)reserve) > 512) c = 2;
      }
    cached[dev].store(c, std::memory_order_relaxed);
  }
  *fit = c == 1;
  return cudaSuccess;
}

bool encode_rows(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* map, const uint8_t* base,
                 int64_t half_k, int64_t rows, int64_t batches, uint32_t box_rows) {
  const cuuint64_t dims[3] = {(cuuint64_t)half_k, (cuuint64_t)rows, (cuuint64_t)batches};
  const cuuint64_t strides[2] = {(cuuint64_t)half_k, (cuuint64_t)(half_k * rows)};
  const cuuint32_t box[3] = {128, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(base), dims, strides, box,
                estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of scale atoms as 8-byte elements: a stage's 2 KB of a row is one box row.
bool encode_atoms(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap* map, const uint8_t* base,
                  int64_t rest_k, int64_t rows, uint32_t box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)(rest_k * 64), (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(rest_k * 512)};
  const cuuint32_t box[2] = {256, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT64, 2, const_cast<uint8_t*>(base), dims, strides, box,
                estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// The dense product's tile and K split, by the time that each would take: rounds of
// tiles over the SMs (or pairs), each its stages or, if longer, the epilogue of the tile
// before, then the last epilogue, in us as measured on GB300.  A stage of a 128 x bn
// tile is bound by its bytes into shared memory.  Rows that do not start on 128-byte
// lines (K % 256 != 0) bring more lines, which costs the more the more SMs ask for them;
// a pair's MMAs nearly hide it.  A last tile with few rows of b brings fewer bytes, and
// fewer columns of the pair's MMAs.  An activation that has an exponential takes the pair
// kernel's epilogue longest.
// Both tiles measured on 366 shapes, 200x9000x544 to 5000x5000x7168, on a part of which
// the constants were fitted: the choice takes 0.2% longer than the faster tile on average
// without an activation, at most 15% (270x2100x5152, 5 batches), and 0.6%, at most 10%,
// with one.  Nearly level choices are where it errs.
GemmChoice choose_gemm(int64_t M, int64_t N, int64_t K, int64_t L, int sms, bool activation) {
  const bool aligned = K % 256 == 0;
  const int64_t stages = (K + 255) / 256, rest_m = (M + 127) / 128;
  struct Kind {
    int bn;
    double stage, tile, epilogue, last_with_activation;
  };
  static constexpr Kind kKinds[] = {{16, 0.20, 0.3, 0.3, 0.7},
                                    {32, 0.21, 0.3, 0.5, 1.1},
                                    {64, 0.22, 0.5, 0.9, 2.0},
                                    {128, 0.30, 0.4, 1.7, 3.8}};
  GemmChoice best = {256, 1};
  const int64_t pair_tiles = L * ((rest_m + 1) / 2) * ((N + 255) / 256), pairs = sms / 2;
  const int64_t pair_rounds = (pair_tiles + pairs - 1) / pairs;
  const int64_t pair_n = (N + 255) / 256, pair_width = N / 256 * 256 + (N % 256 + 63) / 64 * 64;
  const double pair_fill = 0.7 + 0.3 * (double)pair_width / (double)(256 * pair_n);
  const double pair_tile = (double)stages * (aligned ? 0.334 : 0.38) * pair_fill + 1.5;
  double least = (double)(pair_rounds - 1) * std::max(pair_tile, activation ? 6.5 : 3.3) + pair_tile +
                 (activation ? 5.5 : 2.9);
  for (const Kind& k : kKinds) {
    if (k.bn < 128 && N > k.bn) continue;  // a tile starts on a scale atom
    if (k.bn == 128 && N <= 64) continue;  // (the narrower tile was the faster on all of 50 shapes)
    const int64_t tiles_n = (N + k.bn - 1) / k.bn, tiles = L * rest_m * tiles_n;
    const double there = (double)N / (double)(k.bn * tiles_n);
    const double epilogue = activation ? 1.2 * k.epilogue : k.epilogue;
    const double last = activation ? k.last_with_activation : k.epilogue;
    for (int ks = 1; ks <= 4; ks *= 2) {
      // a split needs room for all its CTAs at once, and two stages for each (clusters of
      // 8 start late: 2048x16x8192 took 11.3 us with them, 6.4 with 4, 11.3 without)
      if (ks > 1 && (tiles * ks > sms || stages < 2 * ks)) break;
      const int64_t rounds = (tiles * ks + sms - 1) / sms, own = (stages + ks - 1) / ks;
      double stage = k.stage;
      if (k.bn < 128)
        stage *= aligned ? 1.0 : 1.6;
      else
        stage *= (aligned ? 1.0 : 1.0 + 0.5 * std::min(1.0, (double)(tiles * ks) / sms)) * (0.85 + 0.15 * there);
      const double tile = (double)own * stage + k.tile;
      const double time = (double)(rounds - 1) * std::max(tile, epilogue) + tile + last +
                          (ks > 1 ? 0.8 + 0.02 * k.bn * (ks - 1) : 0.0);
      if (time < least) {
        least = time;
        best = {k.bn, ks};
      }
    }
  }
  return best;
}

cudaError_t launch_gemm(const GemmArgs& g, int sms, cudaStream_t stream) {
  const bool grouped = g.tiles != nullptr;
  GemmParams p;
  memset(&p, 0, sizeof(p));
  p.sfa = g.sfa;
  p.sfb = g.sfb;
  p.tiles = g.tiles;
  p.tile_count = g.tile_count;
  p.c = g.c;
  p.bias = g.bias;
  p.alphas = g.alphas;
  p.q = g.q;
  p.qsf = g.qsf;
  p.M = g.M;
  p.N = g.N;
  p.c_stride = g.c_stride;
  p.alpha = g.alpha;
  p.encode = g.encode;
  p.q_stride = g.M / 4;
  p.q_atom_row = (g.M + 127) / 128 * 512;
  p.c_dtype = g.c_dtype;
  p.activation = g.activation;
  const uintptr_t two = g.c_dtype == kF32 ? 8 : 4;
  p.paired = reinterpret_cast<uintptr_t>(g.c) % two == 0 && g.c_stride % 2 == 0 && g.M % 2 == 0;
  p.rest_m = (int32_t)((g.M + 127) / 128);
  p.rest_n = (int32_t)((g.N + 127) / 128);
  p.rest_k = (int32_t)((g.K + 63) / 64);
  p.kstages = (p.rest_k + 3) / 4;
  if (g.K == 0) {
    p.rows = g.G * g.N;
    const int64_t ctas = (p.rows * g.M + 255) / 256;
    return launch_pdl(gemm_no_k_kernel, dim3((unsigned)(ctas < 16 * sms ? ctas : 16 * sms)), dim3(256),
                      0, stream, p);
  }
  bool fit = false;
  const cudaError_t err = columns_fit_here(&fit);
  if (err != cudaSuccess) return err;
  if (!fit) return cudaErrorNotSupported;
  const GemmChoice choice = grouped ? GemmChoice{g.tile_rows, 1}
                                    : choose_gemm(g.M, g.N, g.K, g.G, sms, g.activation > 1);  // (ReLU costs nothing)
  const int bn = choice.bn;
  const bool pair = bn == 256;
  const int64_t batches = grouped ? 1 : g.G;
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (encode == nullptr) return cudaErrorNotSupported;
  const int64_t half_k = g.K / 2;
  if (!encode_rows(encode, &p.tmap_a, g.a, half_k, g.M, g.G, 128) ||
      !encode_rows(encode, &p.tmap_b, g.b, half_k, g.N, batches, pair ? 128u : (uint32_t)bn))
    return cudaErrorInvalidValue;
  if (pair && (!encode_atoms(encode, &p.tmap_sfa, g.sfa, p.rest_k, g.G * p.rest_m, 1) ||
               !encode_atoms(encode, &p.tmap_sfb, g.sfb, p.rest_k, batches * p.rest_n, 2)))
    return cudaErrorInvalidValue;
  // the pair kernel stores c by TMA (8192 x 8192, K 2048: 53 us, 58 with plain stores;
  // the one-SM kernel's four epilogue warps were slower with it, 58 us against 43 at K 256)
  const int64_t size = g.c_dtype == kF32 ? 4 : 2;
  p.bulk = pair && g.c != nullptr && reinterpret_cast<uintptr_t>(g.c) % 16 == 0 && g.c_stride * size % 16 == 0 &&
           g.c_stride * size * g.N < (int64_t(1) << 40);  // (a tensor map's largest stride)
  if (p.bulk) {
    const cuuint64_t dims[3] = {(cuuint64_t)g.M, (cuuint64_t)g.N, (cuuint64_t)batches};
    const cuuint64_t strides[2] = {(cuuint64_t)(g.c_stride * size), (cuuint64_t)(g.c_stride * size * g.N)};
    const cuuint32_t box[3] = {128, kUnit, 1}, estr[3] = {1, 1, 1};
    const CUtensorMapDataType type = g.c_dtype == kF32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : g.c_dtype == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                          : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    if (encode(&p.tmap_c, type, 3, g.c, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  p.tiles_m = pair ? (p.rest_m + 1) / 2 : p.rest_m;
  if (grouped) {
    p.c_tile_rows = g.compact && bn < 128 ? bn : 0;
    const int64_t max_tiles = g.max_tiles * p.tiles_m;
    return g.q ? launch_for<kGatedQuantize, true>(bn, p, max_tiles, 1, sms, stream)
               : launch_for<kStore, true>(bn, p, max_tiles, 1, sms, stream);
  }
  p.tiles_n = (int32_t)((g.N + bn - 1) / bn);
  p.total = (int32_t)(g.G * p.tiles_n * p.tiles_m);
  return launch_for<kStore, false>(bn, p, p.total, choice.ks, sms, stream);
}

Footprint product_footprint(int tile_rows, bool gated) {
  const int epi = gated ? kGatedQuantize : kStore;
  return tile_rows == 256 ? pair_footprint(epi) : Footprint{gemm_smem_bytes(tile_rows, epi), columns_for(tile_rows)};
}

cudaError_t gemm_wait_timeouts(int reset, int* out) {
  int own = 0, pairs = 0, cache = 0;
  cudaError_t err = cudaMemcpyFromSymbol(&own, g_gemm_timeouts, sizeof(int));
  if (err == cudaSuccess) err = gemm_pair_wait_timeouts(reset, &pairs);
  if (err == cudaSuccess) err = attention_wait_timeouts(reset, &cache);  // (counted with the layer's)
  *out = own + pairs + cache;
  if (err != cudaSuccess || !reset) return err;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_gemm_timeouts, &zero, sizeof(int));
}

}  // namespace nvfp4
