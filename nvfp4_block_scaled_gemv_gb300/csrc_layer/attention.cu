// Attention of a few query tokens per sequence on the 4-bit cache (sm_103a).
//
//   s[t] = scale * q . k[t],  p = exp(s - max s),  out = sum_t p[t] v[t] / sum_t p[t]
//
// over the tokens that a query sees, in one pass over the cache with a running reference for the
// maximum.
//
// Its floor is the cache's bytes: K and V of a token and head are 9/8 D bytes, and the C
// = query tokens x heads of the group columns that share them are few.  So a column
// tile is the N side (8 columns) of the matrix instruction and the cache's tokens the M
// side of S^T = K Q^T, the head's elements the M side of O^T = V^T P^T, which wastes
// nothing on rows that do not exist.  Codes become fp16 in registers: code * scale has 6
// significant bits and is exact, so the only roundings before the fp32 sums are p to fp16
// (2^-11 of itself; below 2^-21 of the row's largest p, 2^-32 of that) and the result's.
//
// A warp works by itself: 32 tokens (D = 64: 64) at a time in a ring of stages that it fills with bulk
// copies, a copy per 16 tokens (a granule of the cache, K and V in one run of bytes).  All
// tiles of all sequences and heads, one after another, are cut into equal runs, one per
// warp, whatever the lengths are; the lengths are read on the device.  A warp that has all
// of an item (a head's columns of one sequence) writes its result.  Of an item that is
// shared, every warp leaves its piece (maximum, sum, unnormalised result); a CTA adds up its warps'
// pieces, and a second small kernel those of CTAs that share an item, in the order of the tokens.
//
// What bounds it.  32 sequences of 16k to 32k tokens, 64 query heads on 8 heads of 128: 160 us, 5.66
// TB/s, 83% of the measured copy (a step of 64 sequences of 8192: 112 us, 80%; 32 heads each with
// its own keys: 403 us, 88%).  A tile of 32 tokens costs a warp ~730 instructions (128 conversions,
// 128 products with scales, 32 MMAs), of the ~800 issue slots that an SM has in the time of its bytes.
// 16 columns take 1.55 times the time of 8 (12 warps, for the registers), heads of 64 1.8 times that of
// their bytes.  Small calls: one sequence of 900 tokens 9.6 us, of which the second kernel is 3 to 4 and lengths,
// page numbers and the first bytes most of the rest, one after the other.
#include <cfloat>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attention.h"
#include "attention_rows.cuh"
#include "layer.h"
#include "ptx.cuh"
#include "ring.h"
#include "tc_ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kMostWarps = 16;
constexpr int64_t kPieceList = (2 * kAttentionCtas * (int64_t)sizeof(int4) + 255) / 256 * 256;

__device__ int g_attention_timeouts;

// Warps of a CTA, as many as the registers take: D * NT / 4 of results, D * NT / 8 of queries, ~65
// beside them (D = 64, NT = 4 with 12 warps spills: 57 us in place of 50 for 16 x 8 query tokens on 8192).
__host__ __device__ constexpr int warps_for(int D, int NT) { return D * NT <= 128 ? 16 : D * NT <= 256 && D != 64 ? 12 : 8; }

template <int D, int NT>
struct Shape {
  static constexpr int kColumns = 8 * NT;
  static constexpr int kPlanes = D / 64;
  static constexpr int kGranule = 2 * kPlanes * kPlaneBytes;  // bytes of K and V of 16 tokens
  // granules of a stage (one costs ~240 instructions beside its granules' own)
  static constexpr int kGranules = D == 64 ? 4 : 2;
  static constexpr int kTile = kGranules * kGranuleTokens;
  static constexpr int kStage = kGranules * kGranule;
  static constexpr int kWarps = warps_for(D, NT);
  static constexpr int kStagesFit = (220 * 1024 / kWarps - 64) / kStage;
  static constexpr int kStages = kStagesFit < 6 ? kStagesFit : 6;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr size_t kSmem = (size_t)kWarps * kStages * (kStage + 8);
  static constexpr int kPiece = kColumns * (D + 2);  // floats: columns of D, then (maximum, sum)
  static_assert(kStages >= 2, "two stages at least");
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same from zero.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Loads of what a bulk copy left in shared memory: through pointers, so that constant distances go
// into the instruction (the waits on the barriers keep them in their place).
__device__ __forceinline__ uint32_t load_32(const uint8_t* p) { return *reinterpret_cast<const uint32_t*>(p); }
__device__ __forceinline__ uint2 load_64(const uint8_t* p) { return *reinterpret_cast<const uint2*>(p); }
// What one lane or some do to a barrier, by a predicate: a branch around it would split the warp.
__device__ __forceinline__ void expect_if(uint32_t bar, uint32_t bytes, bool who) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(
          bar),
      "r"(bytes), "r"((uint32_t)who)
      : "memory");
}
__device__ __forceinline__ void bulk_load_if(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar, bool who) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@p cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar), "r"((uint32_t)who)
      : "memory");
}
// Bits of a where mask, bits of b elsewhere.
__device__ __forceinline__ uint32_t merge_bits(uint32_t a, uint32_t b, uint32_t mask) {
  return (a & mask) | (b & ~mask);
}

// What a sequence asks for: its query tokens, length and tiles.
struct Sequence {
  int32_t n, q0, length;   // query tokens, the first's row, cached tokens (those of the queries among them)
  int32_t first_tile, tiles;
  bool beyond;             // the length is beyond the page table
};

template <int TILE>
__device__ __forceinline__ Sequence sequence_of(const AttentionParams& p, int b) {
  Sequence s;
  const QueryRows rows = query_rows(p, b);
  s.q0 = rows.q0;
  s.n = rows.n;
  s.length = cached_tokens(p, b, s.beyond);
  int32_t lo, hi;
  token_sees(p, s.length, s.n, 0, lo, hi);
  s.first_tile = lo / TILE;
  // (one tile at least, so that somebody writes the result of an empty row)
  s.tiles = s.n == 0 || s.n * p.group > p.few_columns ? 0 : max((s.length + TILE - 1) / TILE - s.first_tile, 1);
  return s;
}

__device__ __forceinline__ int32_t column_tiles(const AttentionParams& p, int32_t n, int columns) {
  return (int32_t)((uint32_t)(n * p.group + columns - 1) / (uint32_t)columns);
}

// The warps' runs of all tiles (fewer than 2^31, the host has seen to that): the first
// `longer` warps have one more than the others.
struct Runs {
  uint32_t each, longer;
  __device__ __forceinline__ uint32_t start(uint32_t w) const { return each * w + min(w, longer); }
  __device__ __forceinline__ uint32_t of(uint32_t tile) const {
    const uint32_t cut = (each + 1) * longer;
    return tile < cut ? tile / (each + 1) : longer + (tile - cut) / each;
  }
};

// The token of a row (0..7) of a matrix instruction's half: the loads of K (rows 0-3 and 4-7
// of a half-warp together) and of V (rows 0, 2, 4, 6 and 1, 3, 5, 7 together) then each touch
// four tokens that are different modulo 4, that is, different banks.
__device__ __forceinline__ int token_of(int row) { return row ^ (row >> 2 & 1); }

// The range of tokens that a column sees.
__device__ __forceinline__ void seen_by(const AttentionParams& p, const Sequence& s, int column, int32_t& lo, int32_t& hi) {
  const int32_t i = column / p.group;  // query token
  lo = hi = 0;
  if (i < s.n) token_sees(p, s.length, s.n, i, lo, hi);
}

template <int D, int NT>
__device__ __forceinline__ void write_columns(const AttentionParams& p, const Sequence& s, int head, int first_column,
                                              const float (&o)[D / 16][NT][4], const float (&m)[NT][2],
                                              const float (&l)[NT][2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const float decode = p.encode_v ? __frcp_rn(ld_now(p.encode_v + head)) : 1.f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int column = first_column + nt * 8 + 2 * q + e;
      const int i = column / p.group;
      if (i >= s.n) continue;
      const int64_t row = (int64_t)(s.q0 + i) * p.Hq + (int64_t)head * p.group + (column - i * p.group);
      const float sum = l[nt][e];
      float f = sum == 0.f ? 0.f : decode / sum;
      if (s.beyond) f = __int_as_float(0x7fc00000);
      if (p.lse != nullptr && g == 0)
        p.lse[row] = s.beyond ? f : sum == 0.f ? -INFINITY : (m[nt][e] + log2f(sum)) * 0.69314718055994531f;
      constexpr int kPer = D == 64 ? 8 : 16;  // elements of a lane in a run
#pragma unroll
      for (int r = 0; r < (D + 127) / 128; ++r) {
        const int64_t at = row * D + r * 128 + g * kPer;
        uint32_t w[kPer / 2];
#pragma unroll
        for (int j = 0; j < kPer / 2; ++j) {
          const float x = o[r * 8 + j][nt][e] * f, y = o[r * 8 + j][nt][2 + e] * f;
          if (p.bf16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
            w[j] = *reinterpret_cast<const uint32_t*>(&h);
          } else {
            w[j] = pack_h2(x, y);
          }
        }
        uint4* const to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at);
#pragma unroll
        for (int j = 0; j < kPer / 8; ++j) to[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
      }
    }
}

// What a warp has of an item that is not all its own: `columns` rows of D unnormalised results,
// and the columns' maxima and sums behind them.
struct Piece {
  const float* at;  // null: none
  Sequence seq;
  uint32_t end;     // the item's end among all tiles
  int32_t head, first_column;
  int32_t early;    // in the workspace, not where the warp's ring was
};

// One more piece of a column, (maximum, sum) and four results, given the maximum of all.
__device__ __forceinline__ void add_piece(float m, float& l, float4& o, float2 ml, float4 v) {
  const float f = ml.x == m ? 1.f : exp2_fast(ml.x - m);
  o.x = fmaf(v.x, f, o.x);
  o.y = fmaf(v.y, f, o.y);
  o.z = fmaf(v.z, f, o.z);
  o.w = fmaf(v.w, f, o.w);
  l = fmaf(ml.y, f, l);
}

// Four results of a column that is all there.
template <int D>
__device__ __forceinline__ void write_four(const AttentionParams& p, const Sequence& s, int head, int column, int d,
                                           float4 o, float m, float l) {
  const int i = column / p.group;
  if (i >= s.n) return;
  const int64_t row = (int64_t)(s.q0 + i) * p.Hq + (int64_t)head * p.group + (column - i * p.group);
  float f = l == 0.f ? 0.f : (p.encode_v ? __frcp_rn(ld_now(p.encode_v + head)) : 1.f) / l;
  if (s.beyond) f = __int_as_float(0x7fc00000);
  if (p.lse != nullptr && d == 0)
    p.lse[row] = s.beyond ? f : l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
  uint2 w;
  if (p.bf16) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(o.x * f, o.y * f), y = __floats2bfloat162_rn(o.z * f, o.w * f);
    w = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  } else {
    w = make_uint2(pack_h2(o.x * f, o.y * f), pack_h2(o.z * f, o.w * f));
  }
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row * D + d) = w;
}

template <int D, int NT>
__global__ void __launch_bounds__(Shape<D, NT>::kThreads, 1) attention_kernel(const AttentionParams p) {
  using S = Shape<D, NT>;
  constexpr int C = S::kColumns, kWarps = S::kWarps, kStages = S::kStages;
  constexpr int kRuns = (D + 127) / 128;           // two planes of V at a time (one, if there is one)
  constexpr int kTilesV = D == 64 ? 4 : 8;         // matrix tiles of a run
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
  const int g = lane >> 2, q = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * kStages * S::kStage;
  const uint32_t bars = smem_u32(smem) + kWarps * kStages * S::kStage + warp * kStages * 8;
  __shared__ uint32_t share_ends[S::kThreads];  // tiles up to the end of each thread's share, in its warp
  __shared__ Piece piece_of[kMostWarps][2];     // that goes on with an item, that begins one

  pdl_launch_dependents();
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) tc::mbar_init(bars + 8 * i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();

  // The tiles of each thread's share of the sequences, their sum, the cut of it into runs, and the
  // sequence that each of this CTA's runs starts in.
  const int share = (p.B + S::kThreads - 1) / S::kThreads;
  const int first_b = threadIdx.x * share;
  uint32_t mine = 0;
  for (int b = first_b; b < min(first_b + share, p.B); ++b) {
    const Sequence seq = sequence_of<S::kTile>(p, b);
    mine += (uint32_t)(seq.tiles * column_tiles(p, seq.n, C));
  }
  mine *= (uint32_t)p.Hkv;
  uint32_t upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += o;
  }
  share_ends[threadIdx.x] = upto;
  if (lane < 2) piece_of[warp][lane].at = nullptr;
  if (threadIdx.x == 0) p.pieces[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
  __syncthreads();
  // (a lane has the sum of a warp's shares)
  uint32_t ends = lane < kWarps ? share_ends[lane * 32 + 31] : 0;
#pragma unroll
  for (int d = 1; d < kWarps; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, ends, d);
    if (lane >= d) ends += o;
  }
  const uint32_t total = __shfl_sync(0xffffffffu, ends, kWarps - 1);
  if (total == 0) return;
  // Warps in use: those of a CTA that are needed for every CTA to have as many, but no fewer than its four
  // schedulers take: a CTA then has more of an item, and fewer pieces are left for the second kernel (1
  // sequence of 400 tokens, 32 heads on 8: 10.0 -> 8.4 us; of 900, 16 heads of 256 on 4: 14.5 -> 11.1;
  // with 6 at least 8.4 and 10.7, but 16 of 100 tokens 9.0 in place of 7.7).
  const uint32_t per_cta = min(max((total + gridDim.x - 1) / gridDim.x, 4u), (uint32_t)kWarps);
  const uint32_t warps = min(per_cta * gridDim.x, total);
  Runs runs;
  runs.each = total / warps;
  runs.longer = total - runs.each * warps;
  const uint32_t cta_rank = blockIdx.x * per_cta, rank = cta_rank + warp;
  bool ok = true;
  if (warp < (int)per_cta && rank < warps) {
  const uint32_t begin = runs.start(rank), end = runs.start(rank + 1);
  // the sequence that the run starts in: its warp of shares, its share, and the place there
  const int chunk = __ffs(__ballot_sync(0xffffffffu, lane < kWarps && begin < ends)) - 1;
  uint32_t before = chunk == 0 ? 0 : __shfl_sync(0xffffffffu, ends, chunk - 1);
  const uint32_t share_end = before + share_ends[chunk * 32 + lane];
  const int place = __ffs(__ballot_sync(0xffffffffu, begin < share_end)) - 1;
  if (place > 0) before = __shfl_sync(0xffffffffu, share_end, place - 1);
  int b = (chunk * 32 + place) * share;
  Sequence seq = sequence_of<S::kTile>(p, b);
  for (;;) {
    const uint32_t here = (uint32_t)(seq.tiles * column_tiles(p, seq.n, C)) * (uint32_t)p.Hkv;
    if (before + here > begin) break;
    before += here;
    seq = sequence_of<S::kTile>(p, ++b);
  }
  // head, column tile and tile at `begin`
  int32_t cts = column_tiles(p, seq.n, C);
  int32_t item = (int32_t)((begin - before) / (uint32_t)seq.tiles);  // head * cts + column tile
  int32_t tile = (int32_t)(begin - before) - item * seq.tiles;

  // the loader: the same walk, some stages ahead
  Sequence ahead = seq;
  int lb = b;
  int32_t litem = item, lcts = cts;
  int32_t ltile = seq.first_tile + tile, ltile_end = seq.first_tile + seq.tiles;  // of the sequence
  uint32_t to_load = end - begin;
  // a lane's granule of the next kWindow tiles, as its number in the cache, or kAbsent (past the
  // length) or kBad (its page does not exist)
  constexpr int64_t kAbsent = -1, kBad = -2;
  constexpr int kGr = S::kGranules, kWindow = 32 / kGr;
  constexpr uint32_t kAll = (1u << kGr) - 1;
  int64_t source = kAbsent;
  int32_t source_tile = ltile - kWindow;
  uint32_t load_stage = 0;
  uint32_t bad_bits = 0;           // kGr bits a stage: granules whose page does not exist
  auto load_next = [&]() {
    if (to_load == 0) return;
    if (ltile >= source_tile + kWindow) {
      source_tile = ltile;
      const int32_t granule = ltile * kGr + lane;
      source = kAbsent;
      if (granule < (ahead.length + kGranuleTokens - 1) / kGranuleTokens) {
        const int32_t page = granule / p.granules;
        const int32_t id = ld_now(p.page_table + (int64_t)lb * p.max_pages + page);
        source = id < 0 || id >= p.pages ? kBad
                                         : ((int64_t)id * p.Hkv + litem / lcts) * p.granules + (granule - page * p.granules);
      }
    }
    const uint32_t bar = bars + 8 * load_stage, dst = ring + load_stage * S::kStage;
    const int64_t mine = __shfl_sync(0xffffffffu, source, (ltile - source_tile) * kGr + (lane & (kGr - 1)));
    const uint32_t valid = __ballot_sync(0xffffffffu, mine >= 0) & kAll;
    const uint32_t bad = __ballot_sync(0xffffffffu, mine == kBad) & kAll;
    expect_if(bar, (uint32_t)__popc(valid) * S::kGranule, lane == 0);
    __syncwarp();
    bulk_load_if(dst + lane * S::kGranule, p.cache + mine * S::kGranule, S::kGranule, bar, (valid >> lane & 1u) != 0);
    bad_bits = (bad_bits & ~(kAll << (kGr * load_stage))) | bad << (kGr * load_stage);
    load_stage = load_stage + 1 == kStages ? 0 : load_stage + 1;
    --to_load;
    if (++ltile == ltile_end && to_load != 0) {
      if (++litem == lcts * p.Hkv) {
        litem = 0;
        do {
          ahead = sequence_of<S::kTile>(p, ++lb);
        } while (ahead.tiles == 0);
        lcts = column_tiles(p, ahead.n, C);
      }
      ltile = ahead.first_tile;
      ltile_end = ltile + ahead.tiles;
      source_tile = ltile - kWindow;
    }
  };
  uint32_t left = end - begin;
  bool primed = false;
  uint32_t stage = 0, parity = 0;
  while (left > 0) {
    // an item, or the part of it in this run
    const int head = item / cts, first_column = (item - head * cts) * C;
    const int32_t from = tile;
    const int32_t to = (uint32_t)(seq.tiles - tile) < left ? seq.tiles : tile + (int32_t)left;

    // its queries: column 8 nt + g, a lane's 16 elements of every plane, as fp16.  bf16
    // values go over in a power of two of the row's own (its largest between 2^14 and 2^15),
    // so that fp16's range is enough; what is then below 2^-39 of the largest is lost.
    uint32_t qf[S::kPlanes][4][2][NT];
    float cs[NT][2];  // score scale of the columns 8 nt + 2 q + e (not 0 or infinite: those times 0 or
                      // an infinity would be NaN)
    const float encode = p.encode_k ? ld_now(p.encode_k + head) : 1.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int column = first_column + nt * 8 + g;
      const int i = column / p.group;
      const bool real = i < seq.n;
      uint32_t w[S::kPlanes][8];
      float largest = 0.f;
      if (real) {
        const uint16_t* const src = static_cast<const uint16_t*>(p.q) + (int64_t)(seq.q0 + i) * p.q_token +
                                    (int64_t)(head * p.group + column - i * p.group) * p.q_head + q * 16;
#pragma unroll
        for (int c = 0; c < S::kPlanes; ++c) {
          const uint4 u = *reinterpret_cast<const uint4*>(src + c * 64), v = *reinterpret_cast<const uint4*>(src + c * 64 + 8);
          w[c][0] = u.x, w[c][1] = u.y, w[c][2] = u.z, w[c][3] = u.w;
          w[c][4] = v.x, w[c][5] = v.y, w[c][6] = v.z, w[c][7] = v.w;
        }
      } else {
#pragma unroll
        for (int c = 0; c < S::kPlanes; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j) w[c][j] = 0u;
      }
      if (nt == 0 && !primed) {
        // (the first queries are on their way)
        primed = true;
#pragma unroll 1
        for (int j = 0; j < kStages; ++j) load_next();
      }
      float back = 1.f;
      if (p.bf16) {
#pragma unroll
        for (int c = 0; c < S::kPlanes; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            largest = fmaxf(largest, fmaxf(fabsf(__uint_as_float(w[c][j] << 16)),
                                           fabsf(__uint_as_float(w[c][j] & 0xffff0000u))));
        largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, 1));
        largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, 2));
        // (zero, infinities and NaN keep an exponent of their own range, and their values)
        const int e = min(max(14 - ((int)(__float_as_uint(largest) >> 23) - 127), -113), 113);
        const float by = __uint_as_float((uint32_t)(e + 127) << 23);
        back = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int c = 0; c < S::kPlanes; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            w[c][j] = pack_h2(__uint_as_float(w[c][j] << 16) * by, __uint_as_float(w[c][j] & 0xffff0000u) * by);
      }
#pragma unroll
      for (int c = 0; c < S::kPlanes; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          qf[c][j][0][nt] = w[c][2 * j];
          qf[c][j][1][nt] = w[c][2 * j + 1];
        }
#pragma unroll
      for (int e = 0; e < 2; ++e)
        cs[nt][e] = fminf(fmaxf(p.scale_log2 * __frcp_rn(encode) * __shfl_sync(0xffffffffu, back, (2 * q + e) * 4), FLT_MIN), FLT_MAX);
    }
    // what the columns see; tiles from full_from to full_to are seen by all of them whole
    int32_t lo[NT][2], hi[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) seen_by(p, seq, first_column + nt * 8 + 2 * q + e, lo[nt][e], hi[nt][e]);
    int32_t full_from, full_to;
    {
      int32_t l0, h0, l1, h1;
      const int last = min(first_column + C, seq.n * p.group) - 1;
      seen_by(p, seq, first_column, l0, h0);
      seen_by(p, seq, last, l1, h1);
      full_from = l1;
      full_to = h0;
    }

    float o[D / 16][NT][4];
    float m[NT][2], l[NT][2];
    // m, or 0 while a row is empty (all its p are 0).  Scores are taken from it before they are scaled: far from 0
    // (scores of 2^28) their product's rounding would be more than the exponential holds.
    float from_m[NT][2];
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][nt][j] = 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) m[nt][e] = -INFINITY, l[nt][e] = from_m[nt][e] = 0.f;

#pragma unroll 1
    for (; tile < to; ++tile) {
      const uint32_t bar = bars + 8 * stage;
      const uint8_t* const base = smem + warp * kStages * S::kStage + stage * S::kStage;
      // (the whole warp waits: one lane's wait under a branch would split it)
      if (!__all_sync(0xffffffffu, tc::mbar_try(bar, parity))) {
        tc::mbar_wait<false>(bar, parity, ok, &g_attention_timeouts);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      const int32_t t0 = (seq.first_tile + tile) * S::kTile;
      const uint32_t bad = bad_bits >> (kGr * stage) & kAll;
      const bool whole = t0 >= full_from && t0 + S::kTile <= full_to && bad == 0;  // (the same in all lanes)

      // S^T, 16 tokens x 8 columns at a time
      const uint8_t* const k_codes = base + token_of(g) * 32 + q * 8;
      const uint8_t* const k_scales = base + kPlaneScales + token_of(g) * 4 + q;
      float s[kGr][NT][4];
#pragma unroll
      for (int i = 0; i < kGr; ++i) {
#pragma unroll
        for (int c = 0; c < S::kPlanes; ++c) {
          const uint8_t* const row = k_codes + i * S::kGranule + c * kPlaneBytes;
          const uint8_t* const scale_at = k_scales + i * S::kGranule + c * kPlaneBytes;
          const uint2 c0 = load_64(row), c1 = load_64(row + 8 * 32);
          const uint32_t s0 = e4m3x2_to_f16x2(scale_at[0] * 0x101u), s1 = e4m3x2_to_f16x2(scale_at[8 * 4] * 0x101u);
          uint32_t a[8], d[8];
          e2m1x8_to_f16x2x4(c0.x, *reinterpret_cast<uint32_t(*)[4]>(&a[0]));
          e2m1x8_to_f16x2x4(c0.y, *reinterpret_cast<uint32_t(*)[4]>(&a[4]));
          e2m1x8_to_f16x2x4(c1.x, *reinterpret_cast<uint32_t(*)[4]>(&d[0]));
          e2m1x8_to_f16x2x4(c1.y, *reinterpret_cast<uint32_t(*)[4]>(&d[4]));
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            a[j] = mul_h2(a[j], s0);
            d[j] = mul_h2(d[j], s1);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (c + j == 0)
                mma_f16_first(s[i][nt], a[0], d[0], a[1], d[1], qf[0][0][0][nt], qf[0][0][1][nt]);
              else
                mma_f16(s[i][nt], a[2 * j], d[2 * j], a[2 * j + 1], d[2 * j + 1], qf[c][j][0][nt], qf[c][j][1][nt]);
            }
        }
      }
      if (!whole) {
#pragma unroll
        for (int i = 0; i < kGr; ++i)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int32_t t = t0 + i * 16 + r * 8 + token_of(g);
            const bool absent = (bad >> i & 1u) != 0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float& v = s[i][nt][2 * r + e];
                if (t < lo[nt][e] || t >= hi[nt][e])
                  v = -INFINITY;
                else if (absent)
                  v = __int_as_float(0x7fc00000);
              }
          }
      }
      // The reference that p is taken from is raised only where a score passes it by 8 (in base
      // 2): p stays below 2^15, results are seldom rescaled, and most tiles ask a vote of the lanes
      // in place of the maximum over them.
      bool passed = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = fmaxf(s[0][nt][e], s[0][nt][2 + e]);
#pragma unroll
          for (int i = 1; i < kGr; ++i) top = fmaxf(fmaxf(top, s[i][nt][e]), s[i][nt][2 + e]);
          // (from -inf any score passes; -inf - -inf is NaN and does not)
          passed |= (top - m[nt][e]) * cs[nt][e] > 8.f;
        }
      if (__any_sync(0xffffffffu, passed)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(s[0][nt][e], s[0][nt][2 + e]);
#pragma unroll
            for (int i = 1; i < kGr; ++i) top = fmaxf(fmaxf(top, s[i][nt][e]), s[i][nt][2 + e]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            if (top > m[nt][e]) {  // (the same in all lanes of a column)
              const float keep = exp2_fast((m[nt][e] - top) * cs[nt][e]);
              m[nt][e] = top;
              from_m[nt][e] = top;
              l[nt][e] *= keep;
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                o[i][nt][e] *= keep;
                o[i][nt][2 + e] *= keep;
              }
            }
          }
      }
      // P, and its transposition to the second product's operand
      uint32_t pf[kGr][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < kGr; ++i)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float p0 = exp2_fast(fmaf(s[i][nt][2 * r] - from_m[nt][0], cs[nt][0], kReferenceP));
            const float p1 = exp2_fast(fmaf(s[i][nt][2 * r + 1] - from_m[nt][1], cs[nt][1], kReferenceP));
            l[nt][0] += p0;
            l[nt][1] += p1;
            pf[i][nt][r] = transpose_8x8(pack_h2(p0, p1));
          }
      }
      // O^T += V^T P^T
      const int t_a = token_of(2 * q), t_b = token_of(2 * q + 1);
      // a lane's block: 16 elements of one of two planes (D = 64: half of one)
      const uint8_t* const v_plane = base + (S::kPlanes + (D == 64 ? 0 : g >> 2)) * kPlaneBytes;
      const uint8_t* const v_codes_a = v_plane + (D == 64 ? g * 4 : (g & 3) * 8) + t_a * 32;
      const uint8_t* const v_codes_b = v_codes_a + (t_b - t_a) * 32;
      const uint8_t* const v_scales_a = v_plane + kPlaneScales + (D == 64 ? g >> 1 : g & 3) + t_a * 4;
      const uint8_t* const v_scales_b = v_scales_a + (t_b - t_a) * 4;
#pragma unroll
      for (int i = 0; i < kGr; ++i)
#pragma unroll
        for (int r = 0; r < kRuns; ++r) {
          constexpr int kScaleStep = 8 * 4, kCodeStep = 8 * 32;
          const int at = i * S::kGranule + 2 * r * kPlaneBytes;
          uint32_t sb[4] = {v_scales_a[at], v_scales_b[at], v_scales_a[at + kScaleStep], v_scales_b[at + kScaleStep]};
          if (!whole) {
            // A masked place adds 0 whatever it holds: tokens past the length and NaN scales
            // become 0, and a NaN goes to the columns that do see its token.
            uint32_t nan = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int32_t t = t0 + i * 16 + (j & 1 ? t_b : t_a) + (j >> 1) * 8;
              if (t >= seq.length || (bad >> i & 1u)) {
                sb[j] = 0;
              } else if ((sb[j] & 0x7Fu) == 0x7Fu) {
                sb[j] = 0;
                nan |= 1u << j;
              }
            }
            if (__any_sync(0xffffffffu, nan != 0)) {
#pragma unroll 1
              for (int other = 0; other < 4; ++other) {
                const uint32_t theirs = __shfl_sync(0xffffffffu, nan, (lane & ~3) | other);
#pragma unroll 1
                for (int j = 0; j < 4; ++j) {
                  const int32_t t = t0 + i * 16 + token_of(2 * other + (j & 1)) + (j >> 1) * 8;
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                      if ((theirs >> j & 1u) && t >= lo[nt][e] && t < hi[nt][e]) {
#pragma unroll
                        for (int x = 0; x < kTilesV; ++x) {
                          o[r * 8 + x][nt][e] = __int_as_float(0x7fc00000);
                          o[r * 8 + x][nt][2 + e] = __int_as_float(0x7fc00000);
                        }
                      }
                }
              }
            }
          }
          const uint32_t s_ab = e4m3x2_to_f16x2(sb[0] | sb[1] << 8), s_cd = e4m3x2_to_f16x2(sb[2] | sb[3] << 8);
          uint32_t codes[4][2];  // the four tokens' codes
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint8_t* const code = (j & 1 ? v_codes_b : v_codes_a) + at + (j >> 1) * kCodeStep;
            if constexpr (D == 64) {
              codes[j][0] = load_32(code);
            } else {
              const uint2 v = load_64(code);
              codes[j][0] = v.x;
              codes[j][1] = v.y;
            }
          }
#pragma unroll
          for (int w = 0; w < kTilesV / 4; ++w) {
            constexpr uint32_t kLow = 0x0F0F0F0Fu;
            // a byte of two tokens' codes of one element: even elements, odd elements
            uint32_t even_ab[4], odd_ab[4], even_cd[4], odd_cd[4];
            e2m1x8_to_f16x2x4(merge_bits(codes[0][w], codes[1][w] << 4, kLow), even_ab);
            e2m1x8_to_f16x2x4(merge_bits(codes[0][w] >> 4, codes[1][w], kLow), odd_ab);
            e2m1x8_to_f16x2x4(merge_bits(codes[2][w], codes[3][w] << 4, kLow), even_cd);
            e2m1x8_to_f16x2x4(merge_bits(codes[2][w] >> 4, codes[3][w], kLow), odd_cd);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t a0 = mul_h2(even_ab[x], s_ab), a1 = mul_h2(odd_ab[x], s_ab);
              const uint32_t a2 = mul_h2(even_cd[x], s_cd), a3 = mul_h2(odd_cd[x], s_cd);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16(o[r * 8 + w * 4 + x][nt], a0, a1, a2, a3, pf[i][nt][0], pf[i][nt][1]);
            }
          }
        }
      __syncwarp();  // the stage has been read
      load_next();
      if (++stage == kStages) stage = 0, parity ^= 1;
    }
    if (!ok) {
      // copies still under way land before the CTA can end
      bool landed = true;
      await_fills(left - (uint32_t)(tile - from), to_load, stage, parity, kStages, [&](uint32_t s, uint32_t of) {
        return tc::mbar_wait<false>(bars + 8 * s, of, landed, &g_attention_timeouts);
      });
      break;
    }
    left -= (uint32_t)(to - from);

    // sums over the lanes that have a column's tokens, and in base 2 what they are relative to
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 4);
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 8);
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 16);
        m[nt][e] = fmaf(m[nt][e], cs[nt][e], -kReferenceP);
      }
    if (from == 0 && to == seq.tiles) {
      write_columns<D, NT>(p, seq, head, first_column, o, m, l);
    } else {
      // A piece.  The run's last one goes where its ring was; one before that, which the ring is
      // still in use beside, to the workspace.
      float* const piece = left == 0 ? reinterpret_cast<float*>(smem + warp * kStages * S::kStage)
                                     : p.partial + ((int64_t)2 * kAttentionCtas + (int64_t)blockIdx.x * kWarps + warp) * S::kPiece;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int column = nt * 8 + 2 * q + e;
          constexpr int kPer = D == 64 ? 8 : 16;
#pragma unroll
          for (int r = 0; r < kRuns; ++r) {
            float* const at = piece + column * D + r * 128 + g * kPer;
#pragma unroll
            for (int j = 0; j < kPer / 4; ++j)
              reinterpret_cast<float4*>(at)[j] = make_float4(o[r * 8 + 2 * j][nt][e], o[r * 8 + 2 * j][nt][2 + e],
                                                             o[r * 8 + 2 * j + 1][nt][e], o[r * 8 + 2 * j + 1][nt][2 + e]);
          }
          if (g == 0) *reinterpret_cast<float2*>(piece + C * D + column * 2) = make_float2(m[nt][e], l[nt][e]);
        }
      if (lane == 0) {
        Piece& to_merge = piece_of[warp][from == 0 ? 1 : 0];
        to_merge.at = piece;
        to_merge.head = head;
        to_merge.first_column = first_column;
        to_merge.early = left != 0;
        to_merge.end = before + (uint32_t)((item + 1) * seq.tiles);
        to_merge.seq = seq;
      }
    }
    // on to the next item
    tile = 0;
    if (left > 0 && ++item == cts * p.Hkv) {
      item = 0;
      do {
        before += (uint32_t)(seq.tiles * cts) * (uint32_t)p.Hkv;
        seq = sequence_of<S::kTile>(p, ++b);
        cts = column_tiles(p, seq.n, C);
      } while (seq.tiles == 0);
    }
  }
  }

  // The CTA's pieces, in the order of its warps: chains of one item each.  Every chain is added up
  // by some warps, into the item's result if it is all there, otherwise into one of the CTA's two
  // places of the workspace: for an item that goes on from the CTA before, and for one that begins
  // here and goes on in the next.  (A CTA with a wait that ran out has none to show.)
  if (__syncthreads_or(!ok)) return;
  const uint32_t present =
      __ballot_sync(0xffffffffu, (lane >> 1) < kWarps && piece_of[min(lane >> 1, kWarps - 1)][lane & 1].at != nullptr);
  if (present == 0) return;
  // (an item begins in the second place of its first warp)
  const uint32_t starts = (present & 0xAAAAAAAAu) | (present & (0u - present));
  const uint32_t cta_end = runs.start(min(cta_rank + per_cta, warps));
  const int chains = __popc(starts);
  const int each = chains < kWarps ? kWarps / chains : 1;  // warps per chain
  for (int chain = warp / each; chain < chains; chain += kWarps / each) {
    uint32_t rest = starts;
    for (int i = 0; i < chain; ++i) rest &= rest - 1;
    const int first = __ffs(rest) - 1;
    rest &= rest - 1;  // of the next chains
    const uint32_t members = present & (0xffffffffu << first) & ((rest & (0u - rest)) - 1u);  // (none: all above)
    const Piece& lead = piece_of[first >> 1][first & 1];
    const bool begins = (first & 1) != 0, ends = lead.end <= cta_end;
    float* const sum_at = p.partial + ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * S::kPiece;
    // pieces where the rings of warps one after another were, and at most one more behind them
    const int last = 31 - __clz(members);
    const bool more = piece_of[last >> 1][last & 1].early != 0;
    const float* const behind = piece_of[last >> 1][last & 1].at;
    const int w0 = first >> 1, w1 = (last >> 1) + (more ? 0 : 1);
    constexpr int kStep = kStages * S::kStage / 4;  // floats from one ring to the next
    const float* const rings = reinterpret_cast<const float*>(smem);
    for (int e = (warp % each) * 32 + lane; e < C * D / 4; e += each * 32) {
      const int c = e / (D / 4), d = e % (D / 4) * 4;
      float l = 0.f, m = more ? behind[C * D + 2 * c] : -INFINITY;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int w = w0; w < w1; ++w) m = fmaxf(m, rings[w * kStep + C * D + 2 * c]);
#pragma unroll 4
      for (int w = w0; w < w1; ++w)
        add_piece(m, l, o, *reinterpret_cast<const float2*>(rings + w * kStep + C * D + 2 * c),
                  *reinterpret_cast<const float4*>(rings + w * kStep + c * D + d));
      if (more)
        add_piece(m, l, o, *reinterpret_cast<const float2*>(behind + C * D + 2 * c),
                  *reinterpret_cast<const float4*>(behind + c * D + d));
      if (begins && ends) {
        write_four<D>(p, lead.seq, lead.head, lead.first_column + c, d, o, m, l);
      } else {
        *reinterpret_cast<float4*>(sum_at + c * D + d) = o;
        if (d == 0) *reinterpret_cast<float2*>(sum_at + C * D + 2 * c) = make_float2(m, l);
      }
    }
    if (begins && !ends && warp % each == 0 && lane == 0) {
      p.pieces[2 * blockIdx.x] = make_int4((int)(runs.of(lead.end - 1) / per_cta), lead.head, lead.first_column, lead.seq.beyond);
      p.pieces[2 * blockIdx.x + 1] = make_int4(lead.seq.n, lead.seq.q0, 0, 0);
    }
  }
}

// The pieces of an item that several CTAs share added up: some CTAs for each CTA of the first
// kernel, for the item that begins in it and goes on in the next, if there is one.  What it takes is
// trips to memory: with all that it has to know of an item written down by the first kernel, one pass
// over the pieces, and the first two fetched at once it is 4 us, where reading lengths and maxima
// first took 6 (4 fetched at once: level).
template <int D, int NT>
__global__ void __launch_bounds__(128) attention_sum_kernel(const AttentionParams p) {
  using S = Shape<D, NT>;
  constexpr int C = S::kColumns;
  pdl_launch_dependents();
  pdl_wait();
  const int e = (int)blockIdx.y * 128 + threadIdx.x;
  const int c = e / (D / 4), d = e % (D / 4) * 4;
  const float* const own = p.partial + (int64_t)blockIdx.x * 2 * S::kPiece;
  // (pieces that are not this item's, or no longer anyone's, are fetched in vain)
  constexpr int kFirst = 2;
  const int4 piece = p.pieces[2 * blockIdx.x], of = p.pieces[2 * blockIdx.x + 1];
  float2 ml[kFirst];
  float4 v[kFirst];
#pragma unroll
  for (int i = 0; i < kFirst; ++i) {
    const float* const at = own + (i == 0 ? S::kPiece : min(i, (int)(gridDim.x - 1 - blockIdx.x)) * 2 * S::kPiece);
    ml[i] = *reinterpret_cast<const float2*>(at + C * D + 2 * c);
    v[i] = *reinterpret_cast<const float4*>(at + c * D + d);
  }
  if (piece.x < 0) return;
  Sequence seq = {};
  seq.n = of.x;
  seq.q0 = of.y;
  seq.beyond = piece.w != 0;
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float2 ml, float4 v) {
    const float top = fmaxf(m, ml.x);
    const float f = m == top ? 1.f : exp2_fast(m - top);
    o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
    l *= f;
    m = top;
    add_piece(m, l, o, ml, v);
  };
  const int count = piece.x - (int)blockIdx.x + 1;
#pragma unroll
  for (int i = 0; i < kFirst; ++i)
    if (i < count) add(ml[i], v[i]);
#pragma unroll 4
  for (int i = kFirst; i < count; ++i) {
    const float* const at = own + (int64_t)i * 2 * S::kPiece;
    add(*reinterpret_cast<const float2*>(at + C * D + 2 * c), *reinterpret_cast<const float4*>(at + c * D + d));
  }
  write_four<D>(p, seq, piece.y, piece.z + c, d, o, m, l);
}

template <int D, int NT>
cudaError_t launch_with(AttentionParams p, void* workspace, int sms, cudaStream_t stream) {
  using S = Shape<D, NT>;
  const int ctas = sms < kAttentionCtas ? sms : kAttentionCtas;
  const cudaError_t err = allow_smem<attention_kernel<D, NT>>(S::kSmem);
  if (err != cudaSuccess) return err;
  p.pieces = static_cast<int4*>(workspace);
  p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kPieceList);
  const cudaError_t ran = launch_pdl(attention_kernel<D, NT>, dim3((unsigned)ctas), dim3(S::kThreads), S::kSmem, stream, p);
  if (ran != cudaSuccess) return ran;
  return launch_pdl(attention_sum_kernel<D, NT>, dim3((unsigned)ctas, S::kColumns * D / 512), dim3(128), 0, stream, p);
}

}  // namespace

int attention_columns(int D, int64_t most) {
  // the fewest columns of a pass that hold a sequence's (the cache is read once), as far as
  // results and queries fit the registers
  const int largest = D >= 128 ? 16 : 32;
  return most <= 8 ? 8 : most <= 16 || largest == 16 ? 16 : 32;
}

int64_t attention_workspace(int D, int columns) {
  const int warps = warps_for(D, columns / 8);
  return kPieceList + (int64_t)kAttentionCtas * (2 + warps) * columns * (D + 2) * 4;
}

cudaError_t launch_attention(AttentionParams p, int D, int columns, void* workspace, int sms, cudaStream_t stream) {
  switch (D * 100 + columns) {
    case 6408: return launch_with<64, 1>(p, workspace, sms, stream);
    case 6416: return launch_with<64, 2>(p, workspace, sms, stream);
    case 6432: return launch_with<64, 4>(p, workspace, sms, stream);
    case 12808: return launch_with<128, 1>(p, workspace, sms, stream);
    case 12816: return launch_with<128, 2>(p, workspace, sms, stream);
    case 25608: return launch_with<256, 1>(p, workspace, sms, stream);
    case 25616: return launch_with<256, 2>(p, workspace, sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t attention_wait_timeouts(int reset, int* out) {
  cudaError_t err = cudaMemcpyFromSymbol(out, g_attention_timeouts, sizeof(int));
  const int zero = 0;
  if (err == cudaSuccess && reset) err = cudaMemcpyToSymbol(g_attention_timeouts, &zero, sizeof(int));
  int prompt = 0;
  if (err == cudaSuccess) err = prompt_wait_timeouts(reset, &prompt);
  *out += prompt;
  return err;
}

}  // namespace nvfp4
