// NVFP4 product on pairs of SMs (tcgen05 cta_group::2, sm_103a): 256 rows of A by
// 256 rows of B per pair; see gemm_tc.cu for the operation.
//
// Why pairs.  A stage (K = 256) of a 128 x 256 tile on one SM brings 54 KB into its
// shared memory for MMAs of ~350 cycles; an SM takes in about 64 bytes per
// cycle, which made that tile 0.40 us per stage (8192^3: 4.35 PFLOP/s).  In a pair
// each SM holds its 128 rows of A and only half of B, the tensor cores read the
// other half from the peer: 38 KB per stage for the same MMAs.
//
// The CTAs of a pair (a cluster of 2) each load their own rows of A and B and
// their scales with TMA, all completing on the leader's barrier; a warp of the
// leader issues the MMAs and another the TMEM copies of the scales, for both CTAs.
// (The 16 instructions of a stage take one issuing thread longer than their
// execution, and more while epilogue warps run beside it.)  Each CTA's accumulator
// (its 128 rows, 256 columns) is in its own tensor memory, and 8 epilogue warps of
// each CTA read it.
//
// What bounds it.  On this kernel's tiles a K = 64 MMA of N = 256 takes 128 cycles (with
// no copies at all a stage took 0.275 us, 9.3 PFLOP/s in all), and the scale copies take
// their turn in the same pipe: 0.33 us per stage, 256 x 256 x 256 per pair.  From one
// tile to the next ~900 cycles pass between the last MMA's commit and the release of
// the shared columns.  Measured on GB300: 8192^3 160 us (6.9 PFLOP/s), 8192 x 8192 with
// K 2048 53 us (5.2), 4096^3 28.7 us (4.8), bf16 c.
//
// A tile of fewer rows of B (the last of an expert, often) runs narrower MMAs, in
// steps of 64: against steps of 128, 385 x 20000 x 8192 43.0 -> 42.1 us and 4000 tokens
// through 6 of 64 experts 373.7 -> 371.0 us; sizes without such a tile the same.
//
// Tensor memory.  Two accumulators of 256 columns and the scales exceed its 512,
// so the accumulators overlap: tile j has columns 0..255 when j is even and
// 112..367 when it is odd.  The epilogue first brings the shared 144 columns into
// registers, and the next tile's MMAs start then, long before it has finished.  The
// scales take three buffers of 48 columns (16 for A, 32 for B), so that a stage's
// copies wait for the MMAs of the third stage before it only, and run beside
// those of the last two.
#include <cstdint>
#include <cstring>

#include "gemm_common.cuh"

namespace nvfp4 {

__device__ int g_gemm_pair_timeouts;

namespace {

using namespace gemm;

constexpr int kPairThreads = 352;  // producer, MMA, scale copies, 8 epilogue warps
constexpr int kEpilogueWarp = 3;   // the first of them
constexpr int kStages = 5;
constexpr uint32_t kBHalf = 128 * 128;
constexpr uint32_t kStageBytes = kABytes + kBHalf + 3 * kAtoms;
constexpr int kBN = 256;
constexpr uint32_t kSecondCol = 112;  // first column of the odd tiles' accumulator
constexpr uint32_t kSfCol = 368, kSfCols = 48;
// units of kUnit columns; the first kFirst of a tile hold all the columns that
// both accumulators have (9 units), and start at kEvenStart in an even tile
constexpr int kUnits = kBN / kUnit, kFirst = 10, kEvenStart = (int)kSecondCol / kUnit;
static_assert(kSecondCol % kUnit == 0 && (kFirst - 1) * kUnit == kBN - (int)kSecondCol, "shared columns");
static_assert(kSecondCol + kBN <= kSfCol && kSfCol + 3 * kSfCols <= 512, "TMEM columns");

constexpr uint32_t pair_smem_bytes(int epi) {
  return kStages * kStageBytes + 1024u + (epi == kGatedQuantize ? 8u * kTransposeBytes : 2u * kStageBytesC);
}
static_assert(most_columns(pair_smem_bytes(kStore), 512) == 512 && most_columns(pair_smem_bytes(kGatedQuantize), 512) == 512,
              "tensor memory of an SM");

// M = 256 over the pair, N = n (see tc::mxf4nvf4_idesc for the fields).
__device__ __forceinline__ uint32_t pair_idesc(uint32_t n) {
  return (1u << 7) | (1u << 10) | ((n >> 3) << 17) | ((256u >> 7) << 27);
}

// TMA loads into this CTA's shared memory that complete on a barrier of either
// CTA of the pair.
__device__ __forceinline__ void pair_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                             uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void pair_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                             uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// Each CTA's own atom (the same shared-memory offset) into its own tensor memory.
__device__ __forceinline__ void pair_copy_atom(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%5], "
      "[%6], p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"((uint32_t)accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}
// Arrive on this barrier of the leader, or of both CTAs, once everything issued
// so far has completed.
__device__ __forceinline__ void pair_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
               : "memory");
}
__device__ __forceinline__ void pair_commit_both(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          bar),
      "h"((uint16_t)3)
      : "memory");
}
// Arrive on a barrier of either CTA without ordering memory: what it announces
// are completed TMEM loads.  (A releasing arrive waits for the warp's stores of
// the tile before, about 1 us.)
__device__ __forceinline__ void arrive_remote_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void pair_alloc(uint32_t slot) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(slot) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_dealloc(uint32_t taddr) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(taddr) : "memory");
}

// N of the MMAs for a tile of so many rows of b: a multiple of 64.
__device__ __forceinline__ int tile_width(int rows) { return (rows + 63) & ~63; }

// Rows of b in tile t (0 past the last tile), the same on every lane.
template <bool GROUPED>
__device__ __forceinline__ int32_t tile_rows_at(const GemmParams& p, int32_t t, int32_t total) {
  return t < total ? __shfl_sync(0xffffffffu, tile_at<kBN, GROUPED>(p, t).rows, 0) : 0;
}

template <int EPI, bool GROUPED>
__global__ void __launch_bounds__(kPairThreads, 1) gemm_pair_kernel(const __grid_constant__ GemmParams p) {
  constexpr int S = kStages;
  extern __shared__ uint8_t pair_smem[];
  __shared__ __align__(8) uint64_t bars[2 * S + 6];
  __shared__ uint32_t tmem_slot;

  const uint32_t raw = smem_u32(pair_smem);
  const uint32_t a_s = (raw + 1023u) & ~1023u;
  const uint32_t b_s = a_s + S * kABytes;
  const uint32_t sfa_s = b_s + S * kBHalf;
  const uint32_t sfb_s = sfa_s + S * kAtoms;
  const uint32_t tr_s = sfb_s + S * 2 * kAtoms;
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int st) { return bar0 + 8u * st; };          // leader's
  auto empty_bar = [&](int st) { return bar0 + 8u * (S + st); };   // each CTA's
  const uint32_t dfull_bar = bar0 + 8u * (2 * S);                  // each CTA's
  const uint32_t dempty_bar = bar0 + 8u * (2 * S + 1);             // leader's
  const uint32_t drain_bar = bar0 + 8u * (2 * S + 2);              // leader's
  auto scale_bar = [&](int i) { return bar0 + 8u * (2 * S + 3 + i); };  // leader's [3]

  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t rank = tc::cluster_rank();
  const int32_t pair = (int32_t)blockIdx.x / 2, pairs = (int32_t)gridDim.x / 2;
  if (threadIdx.x == 0) {
    for (int st = 0; st < S; ++st) {
      tc::mbar_init(full_bar(st), 1);
      tc::mbar_init(empty_bar(st), 1);
    }
    tc::mbar_init(dfull_bar, 1);
    tc::mbar_init(dempty_bar, 16);  // the epilogue warps of both CTAs
    tc::mbar_init(drain_bar, 1);
    for (int i = 0; i < 3; ++i) tc::mbar_init(scale_bar(i), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // the preceding kernels have ended before tensor memory is taken, and the next
  // one may start only after that
  pdl_wait();
  tc::cluster_sync();  // the peer's barriers are initialised, and it is there to allocate
  if (warp == 1) pair_alloc(smem_u32(&tmem_slot));
  tc::fence_before();
  __syncthreads();
  tc::cluster_sync();
  tc::fence_after();
  pdl_launch_dependents();
  constexpr uint32_t tmem = 0;  // (an allocation of all 512 columns starts at the first)
  const int32_t total = GROUPED ? __shfl_sync(0xffffffffu, *p.tile_count, 0) * p.tiles_m : p.total;
  bool ok = true;

  if (warp == 0) {
    int pos = 0, issued = 0;
    uint32_t ph = 0;
    for (int32_t t = pair; t < total; t += pairs) {
      const Tile tile = tile_at<kBN, GROUPED>(p, t);
      const int batch = GROUPED ? 0 : tile.g;
      // the peer's rows of b follow the leader's half of the tile's width
      const int m0 = tile.mt * 256 + (int)rank * 128;
      const int n0 = (int)tile.n0 + (int)rank * (tile_width(tile.rows) / 2);
      // a row tile past the last one reads rows of zeros; its atoms are another's
      const int sa = min(tile.mt * 2 + (int)rank, p.rest_m - 1) + tile.g * p.rest_m;
      const int sb = batch * p.rest_n + (int)(tile.n0 / 128);
      for (int s = 0; s < p.kstages; ++s) {
        tc::mbar_wait<false>(empty_bar(pos), ph ^ 1u, ok, &g_gemm_pair_timeouts);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
          const uint32_t fb = tc::map_rank(full_bar(pos), 0);
          if (elect_one()) {
            // (every box is whole: what is out of range arrives as zeros)
            if (rank == 0) tc::mbar_expect_tx(full_bar(pos), 2 * kStageBytes);
            pair_load_3d(a_s + pos * kABytes, &p.tmap_a, s * 128, m0, tile.g, fb);
            pair_load_3d(b_s + pos * kBHalf, &p.tmap_b, s * 128, n0, batch, fb);
            pair_load_2d(sfa_s + pos * kAtoms, &p.tmap_sfa, s * 256, sa, fb);
            pair_load_2d(sfb_s + pos * 2 * kAtoms, &p.tmap_sfb, s * 256, sb, fb);
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
    // copies still in flight (of both CTAs) land before the CTAs can exit
    if (rank == 0) {
      bool drain_ok = true;
      for (int k = 0; k < S && k < issued; ++k) {
        const int i = issued - 1 - k;
        tc::mbar_wait<false>(full_bar(i % S), (uint32_t)((i / S) & 1), drain_ok, &g_gemm_pair_timeouts);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      const uint64_t da0 = tc::desc_sw128(a_s), db0 = tc::desc_sw128(b_s);
      int pos = 0, j = 0, sf = 0;  // ring slot, tile, scale buffer
      uint32_t ph = 0, sf_ph = 0;
      int32_t rows = tile_rows_at<GROUPED>(p, pair, total);
      for (int32_t t = pair; t < total; t += pairs, ++j) {
        const uint32_t d = tmem + ((j & 1) ? kSecondCol : 0u);
        const uint32_t idesc = pair_idesc((uint32_t)tile_width(rows));
        rows = tile_rows_at<GROUPED>(p, t + pairs, total);  // (the next tile's, ahead of its need)
        // the columns that this tile shares with the one before it have been read
        tc::mbar_wait<false>(dempty_bar, ((uint32_t)j & 1u) ^ 1u, ok, &g_gemm_pair_timeouts);
        for (int s = 0; s < p.kstages; ++s) {
          // the stage's data is here and its scales are in tensor memory
          tc::mbar_wait2(full_bar(pos), ph, scale_bar(sf), sf_ph, ok, &g_gemm_pair_timeouts);
          tc::fence_after();
          const uint32_t ca = tmem + kSfCol + (uint32_t)sf * kSfCols, cb = ca + 16u;
          // (a descriptor counts addresses in units of 16 bytes)
          const uint64_t da = da0 + (uint32_t)pos * (kABytes / 16), db = db0 + (uint32_t)pos * (kBHalf / 16);
          const int nk = p.rest_k - 4 * s;
          __syncwarp();
          if (elect_one() && ok) {
            auto step = [&](int kk, bool accumulate) {
              pair_mma(d, da + 2u * kk, db + 2u * kk, idesc, ca + 4u * kk, cb + 8u * kk, accumulate);
            };
            step(0, s > 0);
            if (nk >= 4) {
              step(1, true);
              step(2, true);
              step(3, true);
            } else {
              if (nk > 1) step(1, true);
              if (nk > 2) step(2, true);
            }
            pair_commit_both(empty_bar(pos));
          }
          __syncwarp();
          if (++sf == 3) {
            sf = 0;
            sf_ph ^= 1u;
          }
          if (++pos == S) {
            pos = 0;
            ph ^= 1u;
          }
        }
        if (elect_one() && ok) pair_commit_both(dfull_bar);
        __syncwarp();
      }
      // every MMA and TMEM copy has finished before tensor memory is released
      if (elect_one()) pair_commit(drain_bar);
      bool drain_ok = true;
      tc::mbar_wait<false>(drain_bar, 0, drain_ok, &g_gemm_pair_timeouts);
      __syncwarp();
    }
  } else if (warp == 2) {
    if (rank == 0) {
      const uint64_t dsa0 = tc::desc_atom(sfa_s), dsb0 = tc::desc_atom(sfb_s);
      int pos = 0, sf = 0;
      uint32_t ph = 0, old_ph = 0;
      int old = -3;  // the slot and phase of the stage three before this one
      int32_t rows = tile_rows_at<GROUPED>(p, pair, total);
      for (int32_t t = pair; t < total; t += pairs) {
        const bool wide = rows > 128;  // scales of a second atom row
        rows = tile_rows_at<GROUPED>(p, t + pairs, total);
        for (int s = 0; s < p.kstages; ++s) {
          // the stage's data is here, and its buffer, last read by the stage three
          // before this one, is free (both barriers asked at once)
          if (old >= 0)
            tc::mbar_wait2(full_bar(pos), ph, empty_bar(old), old_ph, ok, &g_gemm_pair_timeouts);
          else
            tc::mbar_wait<false>(full_bar(pos), ph, ok, &g_gemm_pair_timeouts);
          tc::fence_after();
          const uint32_t ca = tmem + kSfCol + (uint32_t)sf * kSfCols;
          const uint64_t dsa = dsa0 + (uint32_t)pos * (kAtoms / 16), dsb = dsb0 + (uint32_t)pos * (2 * kAtoms / 16);
          const int nk = p.rest_k - 4 * s;
          __syncwarp();
          if (elect_one() && ok) {
            auto step = [&](int kk) {
              pair_copy_atom(ca + 4u * kk, dsa + 32u * kk);
              pair_copy_atom(ca + 16u + 8u * kk, dsb + 32u * kk);
              if (wide) pair_copy_atom(ca + 20u + 8u * kk, dsb + kAtoms / 16 + 32u * kk);
            };
            step(0);
            if (nk >= 4) {
              step(1);
              step(2);
              step(3);
            } else {
              if (nk > 1) step(1);
              if (nk > 2) step(2);
            }
            pair_commit(scale_bar(sf));
          }
          __syncwarp();
          if (++old == S) {
            old = 0;
            old_ph ^= 1u;
          }
          if (++sf == 3) sf = 0;
          if (++pos == S) {
            pos = 0;
            ph ^= 1u;
          }
        }
      }
    }
  } else {
    const int quarter = warp & 3, group = (warp - kEpilogueWarp) >> 2;
    Place w;
    w.transpose = reinterpret_cast<float*>(pair_smem + (tr_s - raw)) +
                  (warp - kEpilogueWarp) * (int)(kTransposeBytes / 4);
    w.staging = tr_s + (uint32_t)group * kStageBytesC;
    w.buffer = 0;
    w.barrier = 1 + group;
    const uint32_t release = tc::map_rank(dempty_bar, 0);
    int j = 0;
    for (int32_t t = pair; t < total; t += pairs, ++j) {
      const Tile tile = tile_at<kBN, GROUPED>(p, t);
      place_at<EPI, GROUPED>(w, p, tile, (int64_t)tile.mt * 2 + rank, quarter);
      if (lane == 0) tc::mbar_wait<false>(dfull_bar, (uint32_t)j & 1u, ok, &g_gemm_pair_timeouts);
      __syncwarp();
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (EPI == kStore) ok = four_warps_all(w.barrier, ok);  // (they meet at it for each unit)
      tc::fence_after();
      const uint32_t d = tmem + ((j & 1) ? kSecondCol : 0u) + ((uint32_t)(32 * quarter) << 16);
      // two groups of four warps take every other unit, the shared columns first:
      // those are all read before any is finished
      const int start = (j & 1) ? 0 : kEvenStart;
      auto column = [&](int i) { return ((start + i) % kUnits) * kUnit; };
      float v[kFirst / 2][kUnit];
      if (ok) {
#pragma unroll
        for (int i = 0; i < kFirst / 2; ++i) tmem_load_16(d + column(2 * i + group), v[i]);
#pragma unroll
        for (int i = 0; i < kFirst / 2; ++i) tmem_wait(v[i]);
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) arrive_remote_relaxed(release);
      if (ok) {
        int n[kFirst / 2];
#pragma unroll
        for (int i = 0; i < kFirst / 2; ++i) n[i] = column(2 * i + group);
        // the others are on their way while these are finished
        constexpr int kRest = (kUnits - kFirst) / 2;
        float rest[kRest][kUnit];
        int rest_n[kRest];
#pragma unroll
        for (int i = 0; i < kRest; ++i) {
          rest_n[i] = column(kFirst + 2 * i + group);
          tmem_load_16(d + rest_n[i], rest[i]);
        }
        finish_columns<EPI, kFirst / 2, true>(p, w, n, v);
#pragma unroll
        for (int i = 0; i < kRest; ++i) tmem_wait(rest[i]);
        finish_columns<EPI, kRest, true>(p, w, rest_n, rest);
      }
    }
    if (EPI == kStore) bulk_wait();
  }

  tc::fence_before();
  __syncthreads();
  tc::cluster_sync();  // neither CTA reads or signals the other's memory any more
  if (warp == 1) {
    tc::fence_after();
    pair_dealloc(tmem);
  }
}

template <int EPI, bool GROUPED>
cudaError_t launch_variant(const GemmParams& p, int64_t max_tiles, int sms, cudaStream_t stream) {
  constexpr auto kern = gemm_pair_kernel<EPI, GROUPED>;
  constexpr uint32_t smem = pair_smem_bytes(EPI);
  cudaError_t err = allow_smem<kern>(smem);
  if (err != cudaSuccess) return err;
  const int64_t pairs = max_tiles < sms / 2 ? max_tiles : sms / 2;
  return launch_pdl(kern, dim3((unsigned)(2 * pairs)), dim3(kPairThreads), smem, stream, p, 2);
}

}  // namespace

cudaError_t launch_gemm_pair(const GemmParams& p, int epi, bool grouped, int64_t max_tiles, int sms,
                             cudaStream_t stream) {
  if (grouped)
    return epi == kGatedQuantize ? launch_variant<kGatedQuantize, true>(p, max_tiles, sms, stream)
                                 : launch_variant<kStore, true>(p, max_tiles, sms, stream);
  return launch_variant<kStore, false>(p, max_tiles, sms, stream);
}

Footprint pair_footprint(int epi) { return {pair_smem_bytes(epi), 512}; }

cudaError_t gemm_pair_wait_timeouts(int reset, int* out) {
  cudaError_t err = cudaMemcpyFromSymbol(out, g_gemm_pair_timeouts, sizeof(int));
  if (err != cudaSuccess || !reset) return err;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_gemm_pair_timeouts, &zero, sizeof(int));
}

}  // namespace nvfp4
