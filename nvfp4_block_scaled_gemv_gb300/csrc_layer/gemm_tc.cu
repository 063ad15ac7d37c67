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
//
// Scale codes are unsigned magnitudes (the MMA ignores bit 7).
//
// Every wait on an mbarrier gives up after tc::kWaitNs, counts a timeout in a
// device word the host can read, and the thread then skips its remaining work.
#include <cstdint>
#include <cstring>

#include "epilogue.cuh"
#include "layer.h"
#include "quantize.cuh"
#include "tc_ptx.cuh"

namespace nvfp4 {

__device__ int g_gemm_timeouts;

namespace {

constexpr int kGemmThreads = 192;
constexpr uint32_t kABytes = 128 * 128;
constexpr uint32_t kAtoms = 4 * 512;  // a stage's scale atoms of 128 rows
constexpr int kTransposePitch = 33;   // floats between columns of a warp's transpose buffer
constexpr int kTransposeCols = 16;

enum Epilogue { kStore = 0, kGatedQuantize = 1 };

__host__ __device__ constexpr uint32_t stage_bytes(int bn) {
  return kABytes + (uint32_t)bn * 128u + kAtoms + (bn > 128 ? 2u : 1u) * kAtoms;
}
__host__ __device__ constexpr int stages_for(int bn) { return bn > 128 ? 4 : bn == 128 ? 5 : 6; }
__host__ __device__ constexpr uint32_t gemm_smem_bytes(int bn, int epi) {
  return (uint32_t)stages_for(bn) * stage_bytes(bn) + 1024u +
         (epi == kGatedQuantize ? 4u * kTransposeCols * kTransposePitch * 4u : 0u);
}

struct GemmParams {
  CUtensorMap tmap_a;  // uint8 {K/2, M, G}, box {128, 128, 1}, 128-byte swizzle
  CUtensorMap tmap_b;  // uint8 {K/2, N, L}, box {128, BN, 1}, 128-byte swizzle
  const uint8_t* sfa;  // [G][rest_m][rest_k][512]
  const uint8_t* sfb;  // [L][rest_n][rest_k][512]
  const int4* tiles;   // grouped: {expert, first row, rows, 0}
  const int32_t* tile_count;
  void* c;
  const float* bias;
  const float* alphas;
  uint8_t* q;
  uint8_t* qsf;
  int64_t M, N, c_stride;
  float alpha, encode;
  int32_t c_dtype, activation;
  int32_t rest_m, rest_n, rest_k, kstages;
  int32_t tiles_n;     // dense: N tiles per batch
  int64_t total;       // dense: tiles
};

// One output tile: rows m0.. of group g's A against rows n0..n0+rows-1 of b.
struct Tile {
  int32_t g;           // batch or expert
  int32_t mt;          // 128-row tile of A
  int64_t n0;          // first row of b (within the batch)
  int32_t rows;        // rows of b in the tile
};

template <int BN, bool GROUPED>
__device__ __forceinline__ Tile tile_at(const GemmParams& p, int64_t t) {
  Tile o;
  const int64_t nt = t / p.rest_m;
  o.mt = (int32_t)(t - nt * p.rest_m);
  if constexpr (GROUPED) {
    const int4 e = p.tiles[nt];
    o.g = e.x;
    o.n0 = e.y;
    o.rows = e.z;
  } else {
    o.g = (int32_t)(nt / p.tiles_n);
    o.n0 = (nt - (int64_t)o.g * p.tiles_n) * BN;
    o.rows = (int32_t)(p.N - o.n0 < BN ? p.N - o.n0 : BN);
  }
  return o;
}

__device__ __forceinline__ void store_c(const GemmParams& p, int64_t idx, float v) {
  if (p.c_dtype == kF32)
    static_cast<float*>(p.c)[idx] = v;
  else if (p.c_dtype == kBF16)
    static_cast<__nv_bfloat16*>(p.c)[idx] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(p.c)[idx] = __float2half_rn(v);
}

template <int BN, int EPI, bool GROUPED>
__global__ void __launch_bounds__(kGemmThreads, 1) gemm_kernel(const __grid_constant__ GemmParams p) {
  constexpr int S = stages_for(BN);
  constexpr int kAcc = BN > 128 ? 1 : 2;            // accumulators in tensor memory
  constexpr uint32_t kSfbAtomRows = BN > 128 ? 2 : 1;
  constexpr uint32_t kSfaCol = kAcc * (BN < 32 ? 32 : BN);
  constexpr uint32_t kSfbCol = kSfaCol + 16 * S;
  static_assert(kSfbCol + 16 * kSfbAtomRows * S <= 512, "TMEM columns");
  extern __shared__ uint8_t gemm_smem[];
  __shared__ __align__(8) uint64_t bars[2 * S + 2 * kAcc + 1];
  __shared__ uint32_t tmem_slot;

  const uint32_t raw = smem_u32(gemm_smem);
  const uint32_t a_s = (raw + 1023u) & ~1023u;
  const uint32_t b_s = a_s + S * kABytes;
  const uint32_t sfa_s = b_s + S * BN * 128u;
  const uint32_t sfb_s = sfa_s + S * kAtoms;
  const uint32_t tr_s = sfb_s + S * kSfbAtomRows * kAtoms;
  uint8_t* const gen = gemm_smem - raw;
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int st) { return bar0 + 8u * st; };
  auto empty_bar = [&](int st) { return bar0 + 8u * (S + st); };
  auto dfull_bar = [&](int i) { return bar0 + 8u * (2 * S + i); };
  auto dempty_bar = [&](int i) { return bar0 + 8u * (2 * S + kAcc + i); };
  const uint32_t drain_bar = bar0 + 8u * (2 * S + 2 * kAcc);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int st = 0; st < S; ++st) {
      tc::mbar_init(full_bar(st), 1);
      tc::mbar_init(empty_bar(st), 1);
    }
    for (int i = 0; i < kAcc; ++i) {
      tc::mbar_init(dfull_bar(i), 1);
      tc::mbar_init(dempty_bar(i), 128);
    }
    tc::mbar_init(drain_bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // the preceding kernels have ended before tensor memory is taken (a kernel
  // that this one waits for may not have taken its own yet), and the next one
  // may start only after that
  pdl_wait();
  if (warp == 1) tc::alloc(smem_u32(&tmem_slot), 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = tmem_slot;
  const int64_t total = GROUPED ? (int64_t)*p.tile_count * p.rest_m : p.total;
  bool ok = true;

  if (warp == 0) {
    if (lane == 0) {
      int pos = 0, issued = 0;
      uint32_t ph = 0;
      for (int64_t t = blockIdx.x; t < total; t += gridDim.x) {
        const Tile tile = tile_at<BN, GROUPED>(p, t);
        const int64_t batch = GROUPED ? 0 : tile.g;
        const uint8_t* sa = p.sfa + ((int64_t)tile.g * p.rest_m + tile.mt) * p.rest_k * 512;
        const uint8_t* sb = p.sfb + (batch * p.rest_n + tile.n0 / 128) * p.rest_k * 512;
        const bool second = BN > 128 && tile.rows > 128;  // the tile has rows in a second atom
        for (int s = 0; s < p.kstages; ++s) {
          const uint32_t nb = (uint32_t)min(4, p.rest_k - 4 * s) * 512u;
          if (tc::mbar_wait<false>(empty_bar(pos), ph ^ 1u, ok, &g_gemm_timeouts)) {
            const uint32_t fb = full_bar(pos);
            tc::mbar_expect_tx(fb, kABytes + BN * 128u + nb * (second ? 3u : 2u));
            tc::tma_load_3d(a_s + pos * kABytes, &p.tmap_a, s * 128, tile.mt * 128, tile.g, fb);
            tc::tma_load_3d(b_s + pos * BN * 128u, &p.tmap_b, s * 128, (int)tile.n0, (int)batch, fb);
            tc::bulk_load(sfa_s + pos * kAtoms, sa + (int64_t)s * kAtoms, nb, fb);
            tc::bulk_load(sfb_s + pos * kSfbAtomRows * kAtoms, sb + (int64_t)s * kAtoms, nb, fb);
            if (second)
              tc::bulk_load(sfb_s + pos * kSfbAtomRows * kAtoms + kAtoms,
                            sb + ((int64_t)p.rest_k + 4 * s) * 512, nb, fb);
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
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = tc::mxf4nvf4_idesc(BN);
      int pos = 0, j = 0;
      uint32_t ph = 0;
      for (int64_t t = blockIdx.x; t < total; t += gridDim.x, ++j) {
        const int acc = j % kAcc;
        const uint32_t d = tmem + acc * BN;
        tc::mbar_wait<false>(dempty_bar(acc), ((uint32_t)(j / kAcc) & 1u) ^ 1u, ok, &g_gemm_timeouts);
        for (int s = 0; s < p.kstages; ++s) {
          const int nk = min(4, p.rest_k - 4 * s);
          if (tc::mbar_wait<false>(full_bar(pos), ph, ok, &g_gemm_timeouts)) {
            tc::fence_after();
            const uint32_t ca = tmem + kSfaCol + 16u * pos, cb = tmem + kSfbCol + 16u * kSfbAtomRows * pos;
            const uint32_t sa = sfa_s + pos * kAtoms, sb = sfb_s + pos * kSfbAtomRows * kAtoms;
            for (int kk = 0; kk < nk; ++kk) {
              tc::copy_atom(ca + 4u * kk, tc::desc_atom(sa + 512u * kk));
              tc::copy_atom(cb + 4u * kSfbAtomRows * kk, tc::desc_atom(sb + 512u * kk));
              if constexpr (BN > 128)
                tc::copy_atom(cb + 8u * kk + 4u, tc::desc_atom(sb + kAtoms + 512u * kk));
            }
            for (int kk = 0; kk < nk; ++kk)
              tc::mma(d, tc::desc_sw128(a_s + pos * kABytes + 32u * kk),
                      tc::desc_sw128(b_s + pos * BN * 128u + 32u * kk), idesc, ca + 4u * kk,
                      cb + 4u * kSfbAtomRows * kk, s > 0 || kk > 0);
            tc::commit(empty_bar(pos));
          }
          if (++pos == S) {
            pos = 0;
            ph ^= 1u;
          }
        }
        if (ok) tc::commit(dfull_bar(acc));
      }
      // every MMA and TMEM copy has finished before TMEM is released
      tc::commit(drain_bar);
      bool drain_ok = true;
      tc::mbar_wait<false>(drain_bar, 0, drain_ok, &g_gemm_timeouts);
    }
    __syncwarp();
  } else {
    const uint32_t quarter = (uint32_t)(warp & 3);
    float* const tr = reinterpret_cast<float*>(gen + tr_s) + (warp - 2) * kTransposeCols * kTransposePitch;
    int j = 0;
    for (int64_t t = blockIdx.x; t < total; t += gridDim.x, ++j) {
      const int acc = j % kAcc;
      const Tile tile = tile_at<BN, GROUPED>(p, t);
      const int64_t m = (int64_t)tile.mt * 128 + 32 * quarter + lane;
      const float alpha = p.alphas ? p.alphas[tile.g] : p.alpha;
      const float bias = p.bias && m < p.M ? p.bias[(int64_t)tile.g * p.M + m] : 0.f;
      if (lane == 0) tc::mbar_wait<false>(dfull_bar(acc), (uint32_t)(j / kAcc) & 1u, ok, &g_gemm_timeouts);
      __syncwarp();
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      constexpr int kCols = EPI == kGatedQuantize ? kTransposeCols : BN < 32 ? 16 : 32;
      if (ok) {
        tc::fence_after();
        for (int n = 0; n < tile.rows; n += kCols) {
          float v[kCols];
          tc::tmem_load_cols<kCols>(tmem + acc * BN + n + ((32u * quarter) << 16), v);
          if constexpr (EPI == kStore) {
            const int64_t row0 = (GROUPED ? 0 : (int64_t)tile.g * p.N) + tile.n0 + n;
            if (m < p.M) {
#pragma unroll
              for (int i = 0; i < kCols; ++i) {
                if (n + i < tile.rows) {
                  float y = fmaf(v[i], alpha, bias);
                  if (p.activation != 0) y = activate(y, p.activation);
                  store_c(p, (row0 + i) * p.c_stride + m, y);
                }
              }
            }
          } else {
            // the quarter's 32 rows are gate and up of 16 outputs: one scale
            // block.  Two lanes take a token, 8 outputs each.
#pragma unroll
            for (int i = 0; i < kCols; ++i) tr[i * kTransposePitch + lane] = v[i];
            __syncwarp();
            const int col = lane >> 1, half = lane & 1;
            float h[8];
            float amax = 0.f;
            bool finite = true;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float gate = tr[col * kTransposePitch + half * 16 + 2 * i] * alpha;
              const float up = tr[col * kTransposePitch + half * 16 + 2 * i + 1] * alpha;
              const float a = p.activation == 2 ? gate / (1.f + expf(-gate)) : activate(gate, p.activation);
              h[i] = a * up * p.encode;
              const float mag = fabsf(h[i]);
              finite = finite && mag < __int_as_float(0x7f800000);
              amax = fmaxf(amax, mag);
            }
            __syncwarp();
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            finite = __shfl_xor_sync(0xffffffffu, finite ? 1 : 0, 1) != 0 && finite;
            uint32_t code = 0x7Fu, q = 0;
            if (finite) {
              float s;
              code = block_scale_code(amax, s);
              if (s > 0.f) q = quantize_8(h, s, 1.0f / s);
            }
            const int64_t row = tile.n0 + n + col;
            const int64_t kb = (int64_t)tile.mt * 4 + quarter;  // scale block of the output row
            const int64_t blocks = p.M / 32, rest = (p.M / 2 + 63) / 64;
            if (n + col < tile.rows) {
              if (kb < blocks)
                *reinterpret_cast<uint32_t*>(p.q + row * (p.M / 4) + kb * 8 + 4 * half) = q;
              if (half == 0 && kb < 4 * rest)
                p.qsf[atom_offset(row, kb, rest)] = kb < blocks ? (uint8_t)code : (uint8_t)0;
            }
          }
        }
      }
      tc::fence_before();
      tc::mbar_arrive(dempty_bar(acc));
    }
  }

  tc::fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after();
    tc::dealloc(tmem, 512);
  }
}

// alpha * 0 + bias for K = 0.
__global__ void __launch_bounds__(256) gemm_no_k_kernel(const GemmParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t total = p.total * p.M;  // rows of all batches * M
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / p.M, m = i - row * p.M;
    float y = p.bias ? p.bias[row / p.N * p.M + m] : 0.f;
    if (p.activation != 0) y = activate(y, p.activation);
    store_c(p, row * p.c_stride + m, y);
  }
}

template <int BN, int EPI, bool GROUPED>
cudaError_t launch_variant(const GemmParams& p, int64_t max_tiles, int sms, cudaStream_t stream) {
  auto kern = gemm_kernel<BN, EPI, GROUPED>;
  const uint32_t smem = gemm_smem_bytes(BN, EPI);
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  const int64_t ctas = max_tiles < sms ? max_tiles : sms;
  return launch_pdl(kern, dim3((unsigned)ctas), dim3(kGemmThreads), smem, stream, p);
}

template <int EPI, bool GROUPED>
cudaError_t launch_bn(int bn, const GemmParams& p, int64_t max_tiles, int sms, cudaStream_t stream) {
  switch (bn) {
    case 16: return launch_variant<16, EPI, GROUPED>(p, max_tiles, sms, stream);
    case 32: return launch_variant<32, EPI, GROUPED>(p, max_tiles, sms, stream);
    case 64: return launch_variant<64, EPI, GROUPED>(p, max_tiles, sms, stream);
    case 128: return launch_variant<128, EPI, GROUPED>(p, max_tiles, sms, stream);
    case 256: return launch_variant<256, EPI, GROUPED>(p, max_tiles, sms, stream);
    default: return cudaErrorInvalidValue;
  }
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

}  // namespace

int gemm_tile_rows(int64_t M, int64_t N, int64_t L, int sms) {
  (void)M; (void)L; (void)sms;
  return N <= 16 ? 16 : N <= 32 ? 32 : N <= 64 ? 64 : N <= 128 ? 128 : 256;
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
  p.c_dtype = g.c_dtype;
  p.activation = g.activation;
  p.rest_m = (int32_t)((g.M + 127) / 128);
  p.rest_n = (int32_t)((g.N + 127) / 128);
  p.rest_k = (int32_t)((g.K + 63) / 64);
  p.kstages = (p.rest_k + 3) / 4;
  if (g.K == 0) {
    p.total = g.G * g.N;
    const int64_t ctas = (p.total * g.M + 255) / 256;
    return launch_pdl(gemm_no_k_kernel, dim3((unsigned)(ctas < 16 * sms ? ctas : 16 * sms)), dim3(256),
                      0, stream, p);
  }
  const int bn = grouped ? g.tile_rows : gemm_tile_rows(g.M, g.N, g.G, sms);
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (encode == nullptr) return cudaErrorNotSupported;
  const int64_t half_k = g.K / 2;
  if (!encode_rows(encode, &p.tmap_a, g.a, half_k, g.M, g.G, 128) ||
      !encode_rows(encode, &p.tmap_b, g.b, half_k, g.N, grouped ? 1 : g.G, (uint32_t)bn))
    return cudaErrorInvalidValue;
  if (grouped) {
    const int64_t max_tiles = g.max_tiles * p.rest_m;
    return g.q ? launch_bn<kGatedQuantize, true>(bn, p, max_tiles, sms, stream)
               : launch_bn<kStore, true>(bn, p, max_tiles, sms, stream);
  }
  p.tiles_n = (int32_t)((g.N + bn - 1) / bn);
  p.total = g.G * p.tiles_n * p.rest_m;
  return launch_bn<kStore, false>(bn, p, p.total, sms, stream);
}

cudaError_t gemm_wait_timeouts(int reset, int* out) {
  cudaError_t err = cudaMemcpyFromSymbol(out, g_gemm_timeouts, sizeof(int));
  if (err != cudaSuccess || !reset) return err;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_gemm_timeouts, &zero, sizeof(int));
}

}  // namespace nvfp4
