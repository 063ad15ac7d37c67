// Attention of many query tokens per sequence on the 4-bit cache, on the tensor cores
// (sm_103a, tcgen05): the same operator as attention.cu, for sequences whose queries and
// heads of a group make more rows than that kernel takes at once.
//
// Its floor is the two products' operations, 4 D per row and token.  A CTA takes 128 NQ rows (query
// tokens x heads of a group, which share the keys) of one sequence and key head, and walks the
// tokens they see in tiles of BN.  The products are tcgen05.mma kind::f16, M = 128:
//
//   S = Q K^T   Q and K in shared memory; S in tensor memory, two buffers
//   O += P V    P in tensor memory, over S's columns or beside them; V in shared memory as it is
//               laid out (its rows are the contraction); O in tensor memory
//
// Four warps turn raw granules into K and V tiles in fp16 (code * scale is exact) in the
// 128-byte swizzled layout that the MMAs read, so that nothing but the 4-bit cache is read from
// memory and nothing dequantised is written there.  Eight warps, a thread per row, do the
// softmax: while one half's rows are worked on, the MMAs of the other half run.  A running
// reference is raised only where a score passes it by 8 (in base 2): p, 2^7 at the reference, then
// stays below 2^15, and the rows of O are seldom rescaled.  p is rounded to fp16 (2^-11 of itself, below
// 2^-21 of the reference's 2^-32 of that), sums are fp32 before that rounding.
//
// Warps: 0-3 and 4-7 softmax of rows 0-127 and 128-255 (NQ = 1: only the first four), 8-11 raw
// tiles to fp16, 12 issues MMAs, 13 copies granules.  Registers are split by what they need: a
// thread of the softmax holds its row's scores of a tile.
//
// Ragged batches know only on the device which sequences are prompts.  A launch has CTAs for the row
// tiles that full ones make and some more; where many short prompts make more than that, a CTA
// takes several, one after the other (a CTA for every row tile there could be: 4096 single tokens and
// a prompt of 2048 took 20 us longer).
//
//   heads of 64    two halves, tiles of 128, P beside S: the next scores need not wait for P's product
//   heads of 128   two halves, tiles of 128, P over S (there is no room beside)
//   heads of 256   rows in plenty: pairs of SMs (CTAS = 2), 128 rows of each, tiles of 128, of which a CTA
//                  brings half the tokens of K and half the elements of V; otherwise one SM, tiles of 64
//
// Heads of 128 on pairs were no faster (1237 against 1202 us when both were measured, 4 prompts of 512 to 4096 tokens after
// prefixes up to 12k, 32 query heads), 64 tokens a tile with P beside S slower (the MMAs of Q K^T read
// 4 KB of Q for 64 columns).
//
// What bounds it.  That case runs at 1.43 PFLOP/s in 1170 us, 75% of the measured bf16 rate, the tensor pipe busy
// about 70% of the time: a half's next scores wait for its softmax and P's product.  Heads of
// 64 run at 0.84 (4 x 2048 queries on 8192 tokens, 575 us): the exponentials and the MMAs of a tile are 1024
// cycles each, and what keeps them from running beside each other is not known.  Heads of 256: 1.09 (2 x 2048 on 8192, 16
// heads, 440 us), for which no cause is known either.
// Short prompts are bound by the beginning and end of a row tile, ~15,000 cycles where 128 tokens are ~2,800: 4 prompts of 2048
// 158 us (189 with rows of Q and results moved a row a lane).
// What mattered most: a wait by one lane under a branch splits the warp for hundreds of cycles, so
// whole warps wait, and single lanes arrive by predicates (1476 -> 1202 us), and a wait that ran out is counted
// when the kernel ends, not in the wait (heads of 64: 655 -> 572 us); one SM's warps share
// 12 KB of the nearest instruction cache with the softmax, so K and V fills are one code, unrolled
// twice (unrolled four times for each of them: 1884 us).
#include <cfloat>
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attention.h"
#include "attention_rows.cuh"
#include "gemm_common.cuh"
#include "layer.h"
#include "ptx.cuh"
#include "quantize.cuh"
#include "tc_ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kPromptThreads = 512;
constexpr uint32_t kPromptColumns = 512;
constexpr int kNanTiles = 4;  // tiles whose NaN marks are kept (more than are in flight)

__device__ int g_prompt_timeouts;

template <int D, int BN, int NQ, int CTAS>
struct Prompt {
  static constexpr int kPlanes = D / 64;
  static constexpr int kRows = 128 * NQ * CTAS;
  static constexpr int64_t kPiece = (int64_t)kRows * (D + 2);  // floats: results, then (reference, sum) of the rows
  static constexpr uint32_t kPanel = 128 * 128;                // a plane of 128 rows of Q
  static constexpr uint32_t kQBytes = (uint32_t)NQ * kPlanes * kPanel;
  // what a CTA has of a tile: some of K's tokens, and some planes of V
  static constexpr int kKeyTokens = BN / CTAS, kValuePlanes = kPlanes / CTAS;
  static constexpr uint32_t kKeyPanel = kKeyTokens * 128, kValuePanel = BN * 128;
  static constexpr uint32_t kSlot = kPlanes * kKeyPanel;
  // raw tiles: K of those tokens, V of all (its scales are looked at for all planes)
  static constexpr uint32_t kSide = kPlanes * kPlaneBytes;  // K or V of a granule
  static constexpr int kKeyGranules = kKeyTokens / kGranuleTokens, kGranules = BN / kGranuleTokens;
  // (one SM: K and V of a granule in one copy, one after the other, as they are in the cache)
  static constexpr int kKeyCopies = CTAS == 1 ? 0 : kKeyGranules, kCopies = kKeyCopies + kGranules;
  static constexpr uint32_t kCopy = CTAS == 1 ? 2 * kSide : kSide, kRaw = kCopies * kCopy;
  static constexpr uint32_t kRawValues = CTAS == 1 ? kSide : kKeyCopies * kSide;  // where V's begin
  static constexpr int kSlots = D == 64 ? 6 : 3;
  static constexpr int kRaws = D == 64 ? 4 : 2;
  // Tensor memory: S, two buffers; P of its own where there is room, otherwise over S; O at the end.
  static constexpr bool kOwnP = NQ == 2 && 3 * BN <= 512 - NQ * D;
  static constexpr uint32_t kS = BN > 128 || kOwnP ? BN : 128, kP = 2 * BN, kO = 512 - NQ * D;
  static_assert(!kOwnP || kP + BN <= kO, "tensor memory");
  static constexpr uint32_t kUsed = 1024 + kQBytes + kSlots * kSlot + kRaws * kRaw + kNanTiles * (BN * 2 + 16);
  static constexpr uint32_t kSmem = kUsed > gemm::kAloneSmem ? kUsed : gemm::kAloneSmem;
  static_assert(kSlot == kValuePlanes * kValuePanel, "a slot holds either");
  static_assert(kCopies <= 32 && kUsed <= 227 * 1024 - 4096, "shared memory");
  static_assert(2 * kNanTiles >= kSlots + 2, "marks of tiles in flight");
};

template <int CTAS>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  if constexpr (CTAS == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
template <int CTAS>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  if constexpr (CTAS == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
// Arrives on this barrier (of both CTAs of a pair) once the MMAs issued so far have completed.
template <int CTAS>
__device__ __forceinline__ void commit_all(uint32_t bar) {
  if constexpr (CTAS == 1)
    tc::commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
// An arrive of some lanes, by a predicate: a branch around it would split the warp.
__device__ __forceinline__ void arrive_if(uint32_t bar, bool who) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %1, 0;\n\t@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
               "r"((uint32_t)who)
               : "memory");
}
// Arrive on the barrier of the CTA that issues the MMAs.  What was written to tensor memory is ordered by tcgen05's own
// fences on both sides, so that its arrive need not order anything;
template <int CTAS>
__device__ __forceinline__ void arrive_issuer(uint32_t bar, bool who) {
  if constexpr (CTAS == 1)
    arrive_if(bar, who);
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %1, 0;\n\t@p mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}" ::"r"(
            tc::map_rank(bar, 0)),
        "r"((uint32_t)who)
        : "memory");
}
// what the warp wrote to (and read of) this CTA's shared memory is released to the cluster first, by a fence of that memory alone (2
// prompts of 2048 on 8192, heads of 256: 441 us; an arrive with a release of its own, of all memory, 541).
template <int CTAS>
__device__ __forceinline__ void arrive_issuer_filled(uint32_t bar, bool who) {
  if constexpr (CTAS == 1) {
    arrive_if(bar, who);
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %1, 0;\n\tfence.release.sync_restrict::shared::cta.cluster;\n\t@p mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}" ::"r"(
            tc::map_rank(bar, 0)),
        "r"((uint32_t)who)
        : "memory");
  }
}
// kind::f16 with fp16 operands and fp32 results; B's rows are the contraction (bit 16).
__host__ __device__ constexpr uint32_t f16_idesc(uint32_t m, uint32_t n, bool b_rows) {
  return (1u << 4) | ((b_rows ? 1u : 0u) << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
}
// A tile whose rows are the contraction: 128-byte rows of 64 elements, 8-row groups 1024 bytes
// apart, the next 64 elements `panel` bytes on.
__device__ __forceinline__ uint64_t desc_rows(uint32_t saddr, uint32_t panel) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(panel >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

#define NVFP4_R32(f) \
  f(0), f(1), f(2), f(3), f(4), f(5), f(6), f(7), f(8), f(9), f(10), f(11), f(12), f(13), f(14), f(15), f(16), \
  f(17), f(18), f(19), f(20), f(21), f(22), f(23), f(24), f(25), f(26), f(27), f(28), f(29), f(30), f(31)

// 32 columns of this warp's lanes, without waiting for them.
__device__ __forceinline__ void tmem_ld_32(uint32_t taddr, uint32_t* v) {
#define NVFP4_OUT(i) "=r"(v[i])
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : NVFP4_R32(NVFP4_OUT)
      : "r"(taddr));
#undef NVFP4_OUT
}
// What was loaded is there (the registers pass through, so that nothing reads them earlier).
__device__ __forceinline__ void tmem_ld_wait(uint32_t* v) {
#define NVFP4_INOUT(i) "+r"(v[i])
  asm volatile("tcgen05.wait::ld.sync.aligned;" : NVFP4_R32(NVFP4_INOUT)::"memory");
#undef NVFP4_INOUT
}
__device__ __forceinline__ void tmem_st_32(uint32_t taddr, const uint32_t* v) {
#define NVFP4_IN(i) "r"(v[i])
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::NVFP4_R32(NVFP4_IN),
      "r"(taddr)
      : "memory");
#undef NVFP4_IN
}
__device__ __forceinline__ void tmem_st_16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15};" ::"r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// tc::mbar_wait for a whole warp, and in line: with a call in it ptxas could not give the warps
// the registers that setmaxnreg asks for.  CTAS 2: arrivals come from the other CTA of the pair too.
template <int CTAS = 1>
__device__ __forceinline__ void wait_phase(uint32_t bar, uint32_t parity, bool& ok) {
  auto done = [&]() { return CTAS == 1 ? tc::mbar_try(bar, parity) : tc::mbar_try_cluster(bar, parity); };
  if (!ok || done()) return;
  const uint64_t t0 = tc::global_ns();
  for (uint32_t i = 1; !done(); ++i)
    if ((i & 63u) == 0 && tc::global_ns() - t0 > tc::kWaitNs) {
      ok = false;
      return;
    }
}
template <int N>
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void async_proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Scores whose row's reference lies further from 0 than this (in base 2) are taken from the reference before they
// are scaled: score * c - round(reference * c), one fused operation elsewhere, is off by half a step of that product,
// 2^-4 here, 1 at 2^24, and from 2^28 more than fp16 (and then the exponential) holds.  (Subtracting first everywhere:
// 1188 us in place of 1172, 4 prompts of up to 4096.)
constexpr float kFarReference = 1048576.f;
// Whether a row's reference m is that far from 0 (-inf: there is none yet).
__device__ __forceinline__ bool is_far(float m, float c) { return fabsf(m * c) > kFarReference && m != -INFINITY; }

__device__ __forceinline__ uint32_t rounded_two(bool bf16, float a, float b) {
  if (!bf16) return pack_h2(a, b);
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// What a CTA works on; the same in all its threads.
struct Work {
  int32_t q0, n, length, head, first_row;  // rows: query token * group + head of the group
  int32_t rows;                            // of the sequence
  int32_t first_token, tiles;              // tokens from first_token, BN at a time
  int32_t full_from, full_to;              // tokens that all its rows see
  int32_t b;
  bool beyond;
};

// What the sum of a row tile's pieces has to know.
struct PieceHead {
  int32_t q0, rows, first_row, beyond;  // rows: 0 if there is no such row tile
};

__device__ __forceinline__ void row_sees(const AttentionParams& p, int32_t length, int32_t n, int32_t row, int32_t& lo,
                                         int32_t& hi) {
  token_sees(p, length, n, row / p.group, lo, hi);
}

// Scores of the tokens t to t + 31 outside [lo, hi) do not count.
__device__ __forceinline__ void mask_32(uint32_t* v, int32_t t, int32_t lo, int32_t hi) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (t + i < lo || t + i >= hi) v[i] = 0xff800000u;
}

template <int BN>
__device__ __forceinline__ bool tile_whole(const Work& w, int32_t t0) {
  return t0 >= w.full_from && t0 + BN <= w.full_to;
}

// Query tokens of a sequence and its first row of q, and the tiles of rows it has here (none,
// if the other kernel takes it).
struct RowTiles : QueryRows {
  int32_t tiles;
};
template <int ROWS>
__device__ __forceinline__ RowTiles row_tiles(const AttentionParams& p, int b) {
  const QueryRows its = query_rows(p, b);
  const int32_t rows = its.n * p.group;
  return {its, rows > p.few_columns ? (rows - 1) / ROWS + 1 : 0};
}

// Ragged batches: row tiles before each sequence, and of all behind them, in one CTA.  (The CTAs
// that find no row tile are told so by one number; each of them counting for itself took 3 us.)
constexpr int kPlanThreads = 1024;
// (Summed in 64 bits: starts that overlap, which nothing forbids the device to hold, then still give
// numbers that only grow, and every row tile that a CTA finds is its sequence's own.)
template <int ROWS>
__global__ void __launch_bounds__(kPlanThreads) attention_prompt_plan_kernel(const AttentionParams p) {
  __shared__ int64_t warp_sums[kPlanThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int share = (p.B + kPlanThreads - 1) / kPlanThreads;
  const int first = min((int)threadIdx.x * share, p.B), end = min(first + share, p.B);
  int64_t mine = 0;
  for (int b = first; b < end; ++b) mine += row_tiles<ROWS>(p, b).tiles;
  int64_t upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == 31) warp_sums[warp] = upto;
  __syncthreads();
  for (int w = 0; w < warp; ++w) upto += warp_sums[w];
  if (threadIdx.x == kPlanThreads - 1) p.row_tiles[p.B] = (int32_t)min(upto, (int64_t)INT32_MAX);
  upto -= mine;
  for (int b = first; b < end; ++b) {
    p.row_tiles[b] = (int32_t)min(upto, (int64_t)INT32_MAX);
    upto += row_tiles<ROWS>(p, b).tiles;
  }
}

template <int D, int BN, int NQ, int CTAS>
__global__ void __launch_bounds__(kPromptThreads, 1) attention_prompt_kernel(const AttentionParams p) {
  using S = Prompt<D, BN, NQ, CTAS>;
  constexpr int kPlanes = S::kPlanes, kSlots = S::kSlots, kRaws = S::kRaws;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kRaws + 2 * kSlots + 10 + kNanTiles];
  __shared__ uint32_t tmem_slot;
  __shared__ uint32_t raw_bad[kRaws];      // granules of a raw tile whose page does not exist
  __shared__ Work shared_work;
  __shared__ uint32_t gave_up;

  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t q_s = base, slot_s = q_s + S::kQBytes, raw_s = slot_s + kSlots * S::kSlot;
  uint8_t* const generic = smem_raw + (base - smem_u32(smem_raw));
  uint16_t* const nan_marks = reinterpret_cast<uint16_t*>(generic + S::kQBytes + kSlots * S::kSlot + kRaws * S::kRaw);
  uint32_t* const nan_any = reinterpret_cast<uint32_t*>(nan_marks + kNanTiles * BN);

  const uint32_t bar0 = smem_u32(bars);
  auto raw_full = [&](int i) { return bar0 + 8u * i; };
  auto raw_empty = [&](int i) { return bar0 + 8u * (kRaws + i); };
  auto slot_full = [&](int i) { return bar0 + 8u * (2 * kRaws + i); };
  auto slot_empty = [&](int i) { return bar0 + 8u * (2 * kRaws + kSlots + i); };
  const uint32_t more = bar0 + 8u * (2 * kRaws + 2 * kSlots);
  const uint32_t q_full = more, drain = more + 8;
  auto s_full = [&](int i) { return more + 16 + 8u * i; };
  auto p_ready = [&](int i) { return more + 32 + 8u * i; };
  // The product of P and V of tile j in half u is through.  Only some tiles' are waited for, and a wait by parity cannot tell
  // a phase from the one two before it: the product before it on the same barrier must be through by then.  With two
  // halves it is, since a half's next scores are asked for after its product; with one half scores are a tile ahead,
  // two products may be under way, and tiles take two barriers in turn.
  auto o_done = [&](int u, int32_t j) { return more + 48 + 8u * (NQ == 2 ? (uint32_t)u : (uint32_t)j & 1u); };
  auto o_phase = [&](int32_t j) { return (uint32_t)(NQ == 2 ? j : j >> 1) & 1u; };
  auto s_free = [&](int i) { return more + 64 + 8u * i; };
  auto marks_full = [&](int i) { return more + 80 + 8u * i; };

  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
  pdl_wait();

  // The CTA's work: row tiles are numbered over the sequences, the last (which sees most) of a
  // sequence first, the key heads of a row tile follow each other, and the parts of its tokens.
  int32_t unit = (int32_t)blockIdx.x / CTAS;
  const int cta = CTAS == 1 ? 0 : (int)tc::cluster_rank();
  const int32_t split = unit % p.splits;
  // (ragged batches: there may be more CTAs than row tiles)
  auto exists = [&](int32_t unit) { return p.row_tiles == nullptr || unit / p.splits / p.Hkv < ld_now(p.row_tiles + p.B); };
  if (!exists(unit)) {
    if (p.splits > 1 && split == 0 && cta == 0 && threadIdx.x == 0)
      reinterpret_cast<PieceHead*>(p.pieces)[unit / p.splits] = {0, 0, 0, 0};
    return;
  }
  // What a unit is, and barriers for it: by one warp.
  auto prepare = [&](int32_t unit, bool again) {
    if (lane == 0) {
      constexpr int kBars = (int)(sizeof(bars) / sizeof(bars[0]));
      if (again)
        for (int i = 0; i < kBars; ++i) asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(bar0 + 8u * i) : "memory");
      for (int i = 0; i < kRaws; ++i) {
        tc::mbar_init(raw_full(i), 1);
        tc::mbar_init(raw_empty(i), 4);
      }
      for (int i = 0; i < kSlots; ++i) {
        tc::mbar_init(slot_full(i), 4 * CTAS);  // the issuer's
        tc::mbar_init(slot_empty(i), 1);
      }
      tc::mbar_init(q_full, 4 * NQ * CTAS);  // the issuer's
      tc::mbar_init(drain, 1);
      for (int i = 0; i < 2; ++i) {
        tc::mbar_init(s_full(i), 1);
        tc::mbar_init(s_free(i), 4 * CTAS);  // the issuer's
        tc::mbar_init(p_ready(i), 4 * CTAS);  // the issuer's
        tc::mbar_init(more + 48 + 8u * i, 1);
      }
      for (int i = 0; i < kNanTiles; ++i) tc::mbar_init(marks_full(i), 4);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    const int32_t item = unit / p.splits, split = unit % p.splits;
    const int32_t rank = item / p.Hkv, head = item % p.Hkv;
    // the last sequence whose row tiles start at or before this one: 32 of them looked at at once
    int b = 0, before = 0;
    if (p.row_tiles == nullptr) {
      const int each = row_tiles<S::kRows>(p, 0).tiles;  // (all alike)
      b = rank / each;
      before = b * each;
    } else {
      for (int end = p.B; end - b > 1;) {
        const int step = (end - b + 31) / 32, at = b + lane * step;
        const bool here = at < end && ld_now(p.row_tiles + at) <= rank;
        b += (__popc(__ballot_sync(0xffffffffu, here)) - 1) * step;
        end = min(end, b + step);
      }
      before = ld_now(p.row_tiles + b);
    }
    if (lane == 0) {
      const RowTiles its = row_tiles<S::kRows>(p, b);
      Work w = {};
      w.q0 = its.q0;
      w.n = its.n;
      w.b = b;
      w.head = head;
      w.rows = w.n * p.group;
      w.first_row = (its.tiles - 1 - (rank - before)) * S::kRows;
      w.length = cached_tokens(p, b, w.beyond);
      const int32_t last_row = min(w.first_row + S::kRows, w.rows) - 1;
      int32_t l0, h0, l1, h1;
      row_sees(p, w.length, w.n, w.first_row, l0, h0);
      row_sees(p, w.length, w.n, last_row, l1, h1);
      w.full_from = l1;
      w.full_to = h0;
      w.first_token = min(l0, max(h1, 0)) / BN * BN;
      w.tiles = max((h1 - w.first_token + BN - 1) / BN, 1);
      const int32_t from = (int32_t)((int64_t)w.tiles * split / p.splits);
      w.tiles = (int32_t)((int64_t)w.tiles * (split + 1) / p.splits) - from;
      w.first_token += from * BN;
      shared_work = w;
      gave_up = 0;
    }
    __syncwarp();
  };
  if (warp == 14) prepare(unit, false);
  __syncthreads();
  float* const piece = p.partial + (int64_t)unit * S::kPiece;
  if (p.splits > 1) {
    if (split == 0 && cta == 0 && threadIdx.x == 0)
      reinterpret_cast<PieceHead*>(p.pieces)[unit / p.splits] = {shared_work.q0, shared_work.rows, shared_work.first_row,
                                                      shared_work.beyond};
    if (shared_work.tiles == 0)  // (fewer tiles than parts)
      for (int i = threadIdx.x; i < S::kRows; i += kPromptThreads)
        reinterpret_cast<float2*>(piece + S::kRows * D)[i] = make_float2(-INFINITY, 0.f);
  }
  if (shared_work.tiles == 0) return;
  // This warp's rows of Q on their way to shared memory, D / 8 lanes to a row: 16-byte copies that hold no
  // registers, in a loop of few instructions (16 loads at once to registers, unrolled, took 4.4 us a
  // row tile for the instructions alone, which are not in the cache when a CTA begins).
  constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
  const int half = warp >> 2, piece16 = lane % kLanes;  // (warps 0 to 7)
  const uint32_t q_panel = q_s + (half * kPlanes + (piece16 >> 3)) * S::kPanel;
  auto query_at = [&](int k) {  // of the warp's k-th rows
    const uint32_t r = (uint32_t)(32 * (warp & 3) + k * kAtOnce + lane / kLanes);
    return q_panel + r * 128 + (uint32_t)((piece16 & 7) ^ (r & 7)) * 16u;
  };
  auto fetch_queries = [&]() {
    const int32_t row = shared_work.first_row + (half * CTAS + cta) * 128 + 32 * (warp & 3) + lane;
    const int32_t token = row / p.group, member = row - token * p.group;
    const int64_t own = row < shared_work.rows ? (int64_t)(shared_work.q0 + token) * p.q_token +
                                                     (int64_t)(shared_work.head * p.group + member) * p.q_head
                                               : -1;
#pragma unroll 4
    for (int k = 0; k < kLanes; ++k) {
      const int64_t from = __shfl_sync(0xffffffffu, own, k * kAtOnce + lane / kLanes);
      const uint16_t* const src = static_cast<const uint16_t*>(p.q) + (from < 0 ? 0 : from) + piece16 * 8;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(query_at(k)), "l"(src), "r"(from < 0 ? 0 : 16)
                   : "memory");
    }
  };
  if (half < NQ) fetch_queries();
  if constexpr (CTAS == 2) tc::cluster_sync();  // the peer's barriers are initialised, and it is there to allocate
  if (warp == 12) {
    if constexpr (CTAS == 1) {
      tc::alloc(smem_u32(&tmem_slot), kPromptColumns);
    } else {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_slot)) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
  }
  // (one SM: the warps that bring tiles begin meanwhile)
  uint32_t tmem = 0;
  if (CTAS == 2 || warp < 8 || warp == 12) {
    tc::fence_before();
    if constexpr (CTAS == 2) {
      __syncthreads();
      tc::cluster_sync();
    } else {
      asm volatile("bar.sync 1, 288;" ::: "memory");
    }
    tc::fence_after();
    tmem = __shfl_sync(0xffffffffu, *const_cast<volatile uint32_t*>(&tmem_slot), 0);
  }
  pdl_launch_dependents();
  bool ok = true;
  // Ragged batches of many sequences on one SM each: the next unit, if there is one.
  auto another = [&]() {
    if constexpr (CTAS == 2) return false;
    unit += (int32_t)gridDim.x;
    if (unit >= p.units || !exists(unit)) return false;
    if (!ok) gave_up = 1;
    tc::fence_before();
    __syncthreads();
    if (gave_up != 0) return false;
    if (warp == 14) prepare(unit, true);
    __syncthreads();
    tc::fence_after();
    return true;
  };

  // Fills of the slots: K of tile j is fill 2 j, V fill 2 j + 1.  Steps x of the products: with two
  // halves tile x / 2 of half x & 1, otherwise tile x; S of a step is buffer x & 1.
  if (warp >= 12) {
    registers_down<56>();
    do {
      const Work work = shared_work;
      const int32_t tiles = work.tiles, steps = tiles * NQ;
      if (warp == 13) {
        // a lane for K or V of a granule
        const int32_t have = (work.length + kGranuleTokens - 1) / kGranuleTokens;
        const bool keys = lane < S::kKeyCopies;
        const int32_t first = work.first_token / kGranuleTokens + (keys ? cta * S::kKeyGranules + lane : lane - S::kKeyCopies);
        int issued = 0;
        auto page_of = [&](int32_t j) {
          const int32_t granule = first + j * S::kGranules;
          if (lane >= S::kCopies || j >= tiles || granule >= have) return INT32_MIN;
          const int32_t id = ld_now(p.page_table + (int64_t)work.b * p.max_pages + granule / p.granules);
          return id >= 0 && id < p.pages ? id : -1;
        };
        int32_t next = page_of(0);
        for (int32_t j = 0; j < tiles && ok; ++j) {
          const int i = j % kRaws;
          const int32_t id = next;
          next = page_of(j + 1);
          wait_phase(raw_empty(i), ((uint32_t)(j / kRaws) & 1u) ^ 1u, ok);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint32_t valid = __ballot_sync(0xffffffffu, id >= 0);
          const uint32_t bad = __ballot_sync(0xffffffffu, id == -1);
          if (lane == 0) {
            raw_bad[i] = bad;
            tc::mbar_expect_tx(raw_full(i), (uint32_t)__popc(valid) * S::kCopy);
          }
          __syncwarp();
          if (id >= 0) {
            const int32_t granule = first + j * S::kGranules;
            const int64_t at = ((int64_t)id * p.Hkv + work.head) * p.granules + granule % p.granules;
            tc::bulk_load(raw_s + i * S::kRaw + lane * S::kCopy, p.cache + (2 * at + (keys || CTAS == 1 ? 0 : 1)) * S::kSide,
                          S::kCopy, raw_full(i));
          }
          ++issued;
        }
        // copies still in flight land before the CTA can exit
        bool landed = true;
        for (int k = 0; k < kRaws && k < issued; ++k) {
          const int i = issued - 1 - k;
          wait_phase(raw_full(i % kRaws), (uint32_t)((i / kRaws) & 1), landed);
        }
        __syncwarp();
      } else if (warp == 12 && cta == 0) {
        constexpr uint32_t qk = f16_idesc(128 * CTAS, BN, false), pv = f16_idesc(128 * CTAS, D, true);
        const uint64_t q_desc = tc::desc_sw128(q_s);
        wait_phase<CTAS>(q_full, 0, ok);
        auto scores = [&](int32_t x) {
          const int32_t j = NQ == 2 ? x >> 1 : x;
          const int u = NQ == 2 ? x & 1 : 0;
          const int fill = 2 * j, i = fill % kSlots;
          wait_phase<CTAS>(slot_full(i), (uint32_t)(fill / kSlots) & 1u, ok);
          ok = __all_sync(0xffffffffu, ok);
          tc::fence_after();
          if (!ok) return;
          const uint64_t a = q_desc + (uint64_t)(u * kPlanes * (S::kPanel >> 4));
          const uint64_t b = tc::desc_sw128(slot_s + i * S::kSlot);
          const uint32_t d = tmem + S::kS * (x & 1);
          if (gemm::elect_one()) {
#pragma unroll
            for (int c = 0; c < kPlanes; ++c)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_ss<CTAS>(d, a + c * (S::kPanel >> 4) + 2 * k, b + c * (S::kKeyPanel >> 4) + 2 * k, qk, c + k > 0);
            commit_all<CTAS>(s_full(x & 1));
            if (u == NQ - 1) commit_all<CTAS>(slot_empty(i));
          }
          __syncwarp();
        };
        scores(0);
        if (steps > 1) scores(1);
        for (int32_t x = 0; x < steps && ok; ++x) {
          if (S::kOwnP && x + 2 < steps) {
            // S is in registers: the next scores need not wait for P and its product
            wait_phase<CTAS>(s_free(x & 1), (uint32_t)(x >> 1) & 1u, ok);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            scores(x + 2);
          }
          const int32_t j = NQ == 2 ? x >> 1 : x;
          const int u = NQ == 2 ? x & 1 : 0;
          const int fill = 2 * j + 1, i = fill % kSlots;
          wait_phase<CTAS>(slot_full(i), (uint32_t)(fill / kSlots) & 1u, ok);
          wait_phase<CTAS>(p_ready(x & 1), (uint32_t)(x >> 1) & 1u, ok);
          ok = __all_sync(0xffffffffu, ok);
          tc::fence_after();
          if (!ok) break;
          const uint64_t b = desc_rows(slot_s + i * S::kSlot, S::kValuePanel);
          const uint32_t a = tmem + (S::kOwnP ? S::kP + (BN / 2) * u : S::kS * (x & 1)), d = tmem + S::kO + D * u;
          if (gemm::elect_one()) {
#pragma unroll
            for (int k = 0; k < BN / 16; ++k)
              mma_ts<CTAS>(d, a + 8u * k, b + (uint64_t)(k * (16 * 128 >> 4)), pv, j > 0 || k > 0);
            commit_all<CTAS>(o_done(u, j));
            if (u == NQ - 1) commit_all<CTAS>(slot_empty(i));
          }
          __syncwarp();
          if (!S::kOwnP && x + 2 < steps) scores(x + 2);
        }
        // every MMA has finished before tensor memory is released
        if (gemm::elect_one()) {
          if constexpr (CTAS == 1)
            tc::commit(drain);
          else
            asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(drain)
                         : "memory");
        }
        bool drained = true;
        wait_phase(drain, 0, drained);
        __syncwarp();
      }
    } while (another());
  } else if (warp >= 8) {
    registers_down<88>();
    do {
      const Work work = shared_work;
      const int32_t tiles = work.tiles;
      // raw granules to fp16 tiles: a warp takes 8 tokens of a plane, a lane a block
      const int w = warp - 8, row8 = lane >> 2, block = lane & 3;
      constexpr int kUnits = S::kKeyTokens / 8 * kPlanes / 4;  // per warp, of either side
      for (int32_t j = 0; j < tiles && ok; ++j) {
        const int ri = j % kRaws;
        const int32_t t0 = work.first_token + j * BN;
        const bool whole = tile_whole<BN>(work, t0);
        wait_phase(raw_full(ri), (uint32_t)(j / kRaws) & 1u, ok);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        __syncwarp();
        const uint32_t bad = raw_bad[ri];
        if (!whole) {
          // Rows that do not see a token must not get a NaN of its V: there the blocks whose scale is
          // NaN become 0, and are marked for the rows that do see them.
          const int t = threadIdx.x - 256;
          uint32_t marks = 0;
          if (t < BN && t0 + t < work.length && !(bad >> (S::kKeyCopies + t / kGranuleTokens) & 1u)) {
            const uint32_t at = raw_s + ri * S::kRaw + S::kRawValues + t / kGranuleTokens * S::kCopy + kPlaneScales +
                                t % kGranuleTokens * 4;
#pragma unroll
            for (int c = 0; c < kPlanes; ++c) {
              uint32_t four;
              asm volatile("ld.shared.b32 %0, [%1];" : "=r"(four) : "r"(at + c * kPlaneBytes));
#pragma unroll
              for (int i = 0; i < 4; ++i) marks |= (four >> (8 * i) & 0x7Fu) == 0x7Fu ? 1u << (4 * c + i) : 0u;
            }
          }
          if (t < BN) nan_marks[j % kNanTiles * BN + t] = (uint16_t)marks;
          const bool any = __any_sync(0xffffffffu, marks != 0);
          if (lane == 0) nan_any[j % kNanTiles * 4 + w] = any;
          __syncwarp();
        }
        arrive_if(marks_full(j % kNanTiles), lane == 0);
        // K, then V: one code for both, with distances that depend on which
#pragma unroll 1
        for (int side = 0; side < 2; ++side) {
          const bool values = side == 1;
          const int own = values ? S::kValuePlanes : kPlanes;  // planes of this CTA
          const uint32_t panel = values ? S::kValuePanel : S::kKeyPanel;
          const int fill = 2 * j + (values ? 1 : 0), si = fill % kSlots;
          wait_phase(slot_empty(si), ((uint32_t)(fill / kSlots) & 1u) ^ 1u, ok);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          __syncwarp();
          const uint32_t from = raw_s + ri * S::kRaw + (values ? S::kRawValues + cta * S::kValuePlanes * kPlaneBytes : 0);
          const uint32_t to = slot_s + si * S::kSlot;
#pragma unroll 2
          for (int k = 0; k < kUnits; ++k) {
            const int unit = w + 4 * k;
            const int group = unit >> (own == 4 ? 2 : own == 2 ? 1 : 0), plane = unit & (own - 1);
            const int t = group * 8 + row8;  // token of this CTA's
            const uint32_t at = from + (group >> 1) * S::kCopy + plane * kPlaneBytes;
            const int row = (group & 1) * 8 + row8;
            uint2 codes;
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(codes.x), "=r"(codes.y) : "r"(at + row * 32 + block * 8));
            uint32_t sb;
            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(sb) : "r"(at + kPlaneScales + row * 4 + block));
            if (!whole || bad) {
              const bool absent = (bad >> ((group >> 1) + (values ? S::kKeyCopies : 0)) & 1u) != 0;
              if (t0 + t + (values ? 0 : cta * S::kKeyTokens) >= work.length || absent) sb = 0;
              if (absent && !values) sb = 0x7Fu;  // its scores are NaN
              if (values && !whole && (sb & 0x7Fu) == 0x7Fu) sb = 0;
            }
            const uint32_t s2 = e4m3x2_to_f16x2(sb * 0x101u);
            uint32_t h[8];
            e2m1x8_to_f16x2x4(codes.x, *reinterpret_cast<uint32_t(*)[4]>(&h[0]));
            e2m1x8_to_f16x2x4(codes.y, *reinterpret_cast<uint32_t(*)[4]>(&h[4]));
#pragma unroll
            for (int i = 0; i < 8; ++i) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h[i]) : "r"(s2));
            // two 16-byte chunks of the token's row, swizzled by the row
            const uint32_t line = to + plane * panel + t * 128;
            const uint32_t c0 = (uint32_t)((2 * block) ^ (t & 7)) * 16u;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(line + c0), "r"(h[0]), "r"(h[1]), "r"(h[2]),
                         "r"(h[3])
                         : "memory");
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(line + (c0 ^ 16u)), "r"(h[4]), "r"(h[5]), "r"(h[6]),
                         "r"(h[7])
                         : "memory");
          }
          async_proxy_fence();
          __syncwarp();
          arrive_issuer_filled<CTAS>(slot_full(si), lane == 0);
          if (values) arrive_if(raw_empty(ri), lane == 0);
        }
      }
    } while (another());
  } else {
    registers_up<184>();
    bool first = true;  // unit of this CTA
    do {
      const Work work = shared_work;
      const int32_t tiles = work.tiles;
      const int u = warp >> 2;
      if (u < NQ) {
        const int r = threadIdx.x & 127;          // row of the half, and lane of tensor memory
        const int in_tile = (u * CTAS + cta) * 128 + r;
        const int32_t row = work.first_row + in_tile;
        const bool real = row < work.rows;
        const int32_t token = row / p.group, member = row - token * p.group;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        // Q as fp16; bf16: in a power of two of the row's own, see attention.cu
        if (!first) fetch_queries();
        first = false;
        asm volatile("cp.async.wait_all;" ::: "memory");
        float back = 1.f;
        if (p.bf16) {
          // (8 pieces at once, all of them what this lane brought: one after the other took 300 cycles each)
#pragma unroll 1
          for (int k0 = 0; k0 < kLanes; k0 += 8) {
            uint32_t words[8][4];
            float largest[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(words[k][0]), "=r"(words[k][1]), "=r"(words[k][2]), "=r"(words[k][3])
                           : "r"(query_at(k0 + k)));
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              largest[k] = 0.f;
#pragma unroll
              for (int i = 0; i < 4; ++i)
                largest[k] = fmaxf(largest[k], fmaxf(fabsf(__uint_as_float(words[k][i] << 16)),
                                                     fabsf(__uint_as_float(words[k][i] & 0xffff0000u))));
            }
#pragma unroll
            for (int d = 1; d < kLanes; d <<= 1)
#pragma unroll
              for (int k = 0; k < 8; ++k) largest[k] = fmaxf(largest[k], __shfl_xor_sync(0xffffffffu, largest[k], d));
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int e = min(max(14 - ((int)(__float_as_uint(largest[k]) >> 23) - 127), -113), 113);
              const float by = __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                words[k][i] = pack_h2(__uint_as_float(words[k][i] << 16) * by, __uint_as_float(words[k][i] & 0xffff0000u) * by);
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(query_at(k0 + k)), "r"(words[k][0]),
                           "r"(words[k][1]), "r"(words[k][2]), "r"(words[k][3])
                           : "memory");
              const int theirs = __shfl_sync(0xffffffffu, e, lane % kAtOnce * kLanes);
              if (lane / kAtOnce == k0 + k) back = __uint_as_float((uint32_t)(127 - theirs) << 23);
            }
          }
        }
        async_proxy_fence();
        __syncwarp();
        arrive_issuer_filled<CTAS>(q_full, lane == 0);

        // (not 0 or infinite: those times 0 or an infinity would be NaN)
        const float decode_k = p.encode_k ? 1.f / ld_now(p.encode_k + work.head) : 1.f;
        const float c = fminf(fmaxf(p.scale_log2 * decode_k * back, FLT_MIN), FLT_MAX);
        int32_t lo, hi;
        row_sees(p, work.length, work.n, real ? row : work.rows - 1, lo, hi);
        float m = -INFINITY;       // the row's reference score, before c
        bool far = false;          // it is far from 0 in some row of the warp
        uint64_t sum = 0;          // two partial sums
        uint32_t nan_blocks = 0;   // blocks of 16 whose V is NaN in a token that the row sees
        const uint32_t o_at = tmem + lanes + S::kO + D * u;
#pragma unroll 1
        for (int32_t j = 0; j < tiles; ++j) {
          const int32_t x = NQ == 2 ? 2 * j + u : j;
          const uint32_t s_at = tmem + lanes + S::kS * (x & 1);
          const uint32_t p_at = S::kOwnP ? tmem + lanes + S::kP + (BN / 2) * u : s_at;
          const int32_t t0 = work.first_token + j * BN;
          wait_phase(s_full(x & 1), (uint32_t)(x >> 1) & 1u, ok);
          ok = __all_sync(0xffffffffu, ok);
          __syncwarp();
          if (!ok) break;
          tc::fence_after();
          const bool whole = tile_whole<BN>(work, t0);
          uint32_t s[BN / 32][32];
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int h = 0; h < BN / 32; ++h) tmem_ld_32(s_at + 32 * h, s[h]);
#pragma unroll
          for (int h = 0; h < BN / 32; ++h) {
            uint32_t* const v = s[h];
            tmem_ld_wait(v);
            if (!whole) mask_32(v, t0 + 32 * h, lo, hi);
#pragma unroll
            for (int i = 0; i < 32; i += 8)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                top[k] = fmaxf(fmaxf(top[k], __uint_as_float(v[i + 2 * k])), __uint_as_float(v[i + 2 * k + 1]));
          }
          if constexpr (S::kOwnP) {
            tc::fence_before();
            __syncwarp();
            arrive_issuer<CTAS>(s_free(x & 1), lane == 0);
            // the product before this one has read its P (and O may be rescaled)
            if (j > 0) {
              wait_phase(o_done(u, j - 1), o_phase(j - 1), ok);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              tc::fence_after();
            }
          }
          const float now = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
          // (from -inf any score passes)
          const bool up = (now - m) * c > 8.f || (m == -INFINITY && now > m);
          if (__any_sync(0xffffffffu, up)) {
            const float f = up ? (m == -INFINITY ? 0.f : exp2_fast((m - now) * c)) : 1.f;
            if (up) m = now;
            const float2 two = unpack_f32x2(sum);
            sum = pack_f32x2(two.x * f, two.y * f);
            far = __any_sync(0xffffffffu, is_far(m, c));
            if (j > 0) {
              if (!S::kOwnP) {
                wait_phase(o_done(u, j - 1), o_phase(j - 1), ok);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc::fence_after();
              }
#pragma unroll 1
              for (int i = 0; i < D; i += 32) {
                uint32_t o[32];
                tmem_ld_32(o_at + i, o);
                tmem_ld_wait(o);
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                tmem_st_32(o_at + i, o);
              }
            }
          }
          float base2 = m == -INFINITY ? 0.f : fmaf(-m, c, kReferenceP);
          if (far) {
            const float less = is_far(m, c) ? m : 0.f;
#pragma unroll
            for (int h = 0; h < BN / 32; ++h)
#pragma unroll
              for (int i = 0; i < 32; ++i) s[h][i] = __float_as_uint(__uint_as_float(s[h][i]) - less);
            if (is_far(m, c)) base2 = kReferenceP;
          }
          const uint64_t c2 = pack_f32x2(c, c), b2 = pack_f32x2(base2, base2), one2 = pack_f32x2(1.f, 1.f);
          uint64_t other = 0;
#pragma unroll
          for (int h = 0; h < BN / 32; ++h) {
            const uint32_t* const v = s[h];
            uint32_t packed[16];
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              float2 a = unpack_f32x2(fma2(pack_f32x2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), c2, b2));
              float2 b = unpack_f32x2(fma2(pack_f32x2(__uint_as_float(v[i + 2]), __uint_as_float(v[i + 3])), c2, b2));
              a.x = exp2_fast(a.x), a.y = exp2_fast(a.y), b.x = exp2_fast(b.x), b.y = exp2_fast(b.y);
              sum = fma2(pack_f32x2(a.x, a.y), one2, sum);
              other = fma2(pack_f32x2(b.x, b.y), one2, other);
              packed[i / 2] = pack_h2(a.x, a.y);
              packed[i / 2 + 1] = pack_h2(b.x, b.y);
            }
            tmem_st_16(p_at + 16 * h, packed);
          }
          sum = fma2(other, one2, sum);
          if (!whole) {
            // (before P is handed over: the marks' place is not used again until then)
            const int marks = j % kNanTiles;
            wait_phase(marks_full(marks), (uint32_t)(j / kNanTiles) & 1u, ok);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            __syncwarp();
            if ((nan_any[marks * 4] | nan_any[marks * 4 + 1] | nan_any[marks * 4 + 2] | nan_any[marks * 4 + 3]) != 0)
              for (int i = 0; i < BN; ++i)
                if (t0 + i >= lo && t0 + i < hi) nan_blocks |= nan_marks[marks * BN + i];
          }
          tmem_st_wait();
          tc::fence_before();
          __syncwarp();
          if (CTAS == 1 || whole)
            arrive_issuer<CTAS>(p_ready(x & 1), lane == 0);
          else  // (the marks have been read)
            arrive_issuer_filled<CTAS>(p_ready(x & 1), lane == 0);
        }
        wait_phase(o_done(u, tiles - 1), o_phase(tiles - 1), ok);
        ok = __all_sync(0xffffffffu, ok);
        __syncwarp();
        tc::fence_after();
        const float2 two = unpack_f32x2(sum);
        const float l = two.x + two.y, relative_to = fmaf(m, c, -kReferenceP);  // (-inf: nothing)
        const float decode = p.encode_v ? 1.f / ld_now(p.encode_v + work.head) : 1.f;
        float f = l == 0.f ? 0.f : decode / l;
        if (work.beyond) f = __int_as_float(0x7fc00000);
        const int64_t out_row = (int64_t)(work.q0 + token) * p.Hq + (int64_t)work.head * p.group + member;
        const bool part = p.splits > 1;
        if (part) {
          f = 1.f;
          if (ok) reinterpret_cast<float2*>(piece + S::kRows * D)[in_tile] = make_float2(relative_to, l);
        } else if (ok && real && p.lse != nullptr) {
          p.lse[out_row] = work.beyond ? f : l == 0.f ? -INFINITY : (relative_to + log2f(l)) * 0.69314718055994531f;
        }
#pragma unroll 1
        for (int i = 0; i < D && ok; i += 32) {
          uint32_t o[32];
          tmem_ld_32(o_at + i, o);
          tmem_ld_wait(o);
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const float g = nan_blocks >> (i / 16 + k / 16) & 1u ? __int_as_float(0x7fc00000) : f;
            o[k] = __float_as_uint(__uint_as_float(o[k]) * g);
          }
          if (part) {
            uint4* const to = reinterpret_cast<uint4*>(piece + (int64_t)in_tile * D + i);
#pragma unroll
            for (int k = 0; k < 8; ++k) to[k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          } else {
            // to where the row of Q was: its products are through
            const uint32_t line = q_s + (half * kPlanes + (i >> 6)) * S::kPanel + r * 128;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t words[4];
#pragma unroll
              for (int x = 0; x < 4; ++x)
                words[x] = rounded_two(p.bf16, __uint_as_float(o[8 * k + 2 * x]), __uint_as_float(o[8 * k + 2 * x + 1]));
              const uint32_t at = line + (uint32_t)((((i & 63) >> 3) + k) ^ (r & 7)) * 16u;
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(words[0]), "r"(words[1]), "r"(words[2]),
                           "r"(words[3])
                           : "memory");
            }
          }
        }
        if (!part && ok) {
          // whole rows out, D / 8 lanes to each (a row a lane: 32 pieces of 16 bytes a store)
          __syncwarp();
          const int64_t own = real ? out_row : -1;
#pragma unroll 4
          for (int k = 0; k < kLanes; ++k) {
            const int64_t to = __shfl_sync(0xffffffffu, own, k * kAtOnce + lane / kLanes);
            uint4 v;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(query_at(k)));
            if (to >= 0) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + to * D + piece16 * 8) = v;
          }
        }
      }
    } while (another());
  }
  if (!ok && lane == 0) atomicAdd(&g_prompt_timeouts, 1);
  tc::fence_before();
  __syncthreads();
  if constexpr (CTAS == 2) tc::cluster_sync();  // neither CTA reads or signals the other's memory any more
  if (warp == 12) {
    tc::fence_after();
    if constexpr (CTAS == 1)
      tc::dealloc(tmem, kPromptColumns);
    else
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// The parts of a row tile added up, in the order of the tokens: 256 threads, four results each.
template <int D, int BN, int NQ, int CTAS>
__global__ void __launch_bounds__(256) attention_prompt_sum_kernel(const AttentionParams p) {
  using S = Prompt<D, BN, NQ, CTAS>;
  pdl_launch_dependents();
  pdl_wait();
  const PieceHead at = reinterpret_cast<const PieceHead*>(p.pieces)[blockIdx.x];
  const int r = (int)(blockIdx.y * 256 + threadIdx.x) / (D / 4), d = threadIdx.x % (D / 4) * 4;
  const int32_t row = at.first_row + r;
  if ((uint32_t)row >= (uint32_t)at.rows) return;
  const float* const pieces = p.partial + (int64_t)blockIdx.x * p.splits * S::kPiece;
  float m = -INFINITY, l = 0.f;
#pragma unroll 4
  for (int i = 0; i < p.splits; ++i) m = fmaxf(m, pieces[i * S::kPiece + S::kRows * D + 2 * r]);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < p.splits; ++i) {
    const float* const piece = pieces + i * S::kPiece;
    const float2 ml = *reinterpret_cast<const float2*>(piece + S::kRows * D + 2 * r);
    const float4 v = *reinterpret_cast<const float4*>(piece + (int64_t)r * D + d);
    if (ml.y == 0.f) continue;  // (nothing that the row sees; a part without tiles has no results at all)
    const float f = ml.x == m ? 1.f : exp2_fast(ml.x - m);
    o.x = fmaf(v.x, f, o.x);
    o.y = fmaf(v.y, f, o.y);
    o.z = fmaf(v.z, f, o.z);
    o.w = fmaf(v.w, f, o.w);
    l = fmaf(ml.y, f, l);
  }
  const int head = (int)blockIdx.x % p.Hkv;
  const int32_t token = row / p.group, member = row - token * p.group;
  const int64_t out_row = (int64_t)(at.q0 + token) * p.Hq + (int64_t)head * p.group + member;
  float f = l == 0.f ? 0.f : (p.encode_v ? 1.f / ld_now(p.encode_v + head) : 1.f) / l;
  if (at.beyond) f = __int_as_float(0x7fc00000);
  if (p.lse != nullptr && d == 0)
    p.lse[out_row] = at.beyond ? f : l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + out_row * D + d) =
      make_uint2(rounded_two(p.bf16, o.x * f, o.y * f), rounded_two(p.bf16, o.z * f, o.w * f));
}

// Row tiles of all sequences: in ragged batches at most (every sequence that has some begins one
// more than its rows fill).
int64_t most_row_tiles(const AttentionParams& p, int rows_per_tile) {
  const int64_t rows = (int64_t)p.T * p.group, sequences = rows / (p.few_columns + 1);
  if (!p.ragged) return (int64_t)p.B * ((rows / p.B + rows_per_tile - 1) / rows_per_tile);
  return rows / rows_per_tile + (sequences < p.B ? sequences : p.B);
}

int64_t round_up(int64_t bytes) { return (bytes + 255) / 256 * 256; }

// Parts that the tokens of a row tile are cut into: as many as bring the row tiles and heads to the
// SMs, where these are fewer, but at most twice the SMs in all, and 4 tiles a part of the tokens that the page table
// has room for.  The lengths are on the device, and a window is not looked at: where the table is wider than the
// sequences, or a window narrower, parts are shorter than that, and some have no tile (512 tokens of 8 heads on one, in a
// table for 131072: 8 parts).
int prompt_splits(int64_t items, int64_t most_tokens, int tile, int ctas) {
  const int64_t places = kAttentionCtas / ctas;
  if (items >= places) return 1;
  const int64_t long_enough = most_tokens / (4 * tile);
  int best = 1;
  double least = 1e30;
  for (int64_t s = 1; s * items <= 2 * places && (s == 1 || s <= long_enough); ++s) {
    const double rounds = (double)((s * items + places - 1) / places) / (double)s + 0.01 * (double)s;
    if (rounds < least) least = rounds, best = (int)s;
  }
  return best;
}

// The launch's sizes, and where in the workspace its parts lie: row tiles of sequences (ragged
// batches), heads of pieces, pieces.
struct PromptPlan {
  int64_t items, heads_at, pieces_at, bytes;
  int64_t ctas;  // (or pairs)
  int splits;
};
template <int D, int BN, int NQ, int CTAS>
PromptPlan plan_with(const AttentionParams& p) {
  using S = Prompt<D, BN, NQ, CTAS>;
  PromptPlan plan;
  plan.items = most_row_tiles(p, S::kRows) * p.Hkv;
  plan.splits = prompt_splits(plan.items, p.capacity, BN, CTAS);
  // Row tiles that only many short prompts have are taken by CTAs that are through with others.
  const int64_t full = ((int64_t)p.T * p.group / S::kRows + 1) * p.Hkv + 2 * kAttentionCtas;
  plan.ctas = CTAS == 1 && p.ragged && plan.splits == 1 && full < plan.items ? full : plan.items * plan.splits;
  plan.heads_at = p.ragged ? round_up(((int64_t)p.B + 1) * 4) : 0;
  plan.pieces_at = plan.heads_at + (plan.splits > 1 ? round_up(plan.items * (int64_t)sizeof(PieceHead)) : 0);
  plan.bytes = plan.pieces_at + (plan.splits > 1 ? plan.items * plan.splits * S::kPiece * 4 : 0);
  return plan;
}

template <int D, int BN, int NQ, int CTAS>
cudaError_t launch_with(AttentionParams p, void* workspace, cudaStream_t stream) {
  using S = Prompt<D, BN, NQ, CTAS>;
  cudaError_t err = allow_smem<attention_prompt_kernel<D, BN, NQ, CTAS>>(S::kSmem);
  if (err != cudaSuccess) return err;
  const PromptPlan plan = plan_with<D, BN, NQ, CTAS>(p);
  uint8_t* const base = static_cast<uint8_t*>(workspace);
  p.splits = plan.splits;
  p.units = (int32_t)(plan.items * plan.splits);
  p.row_tiles = p.ragged ? reinterpret_cast<int32_t*>(base) : nullptr;
  p.pieces = reinterpret_cast<int4*>(base + plan.heads_at);
  p.partial = reinterpret_cast<float*>(base + plan.pieces_at);
  if (p.ragged) {
    err = launch_pdl(attention_prompt_plan_kernel<S::kRows>, dim3(1), dim3(kPlanThreads), 0, stream, p);
    if (err != cudaSuccess) return err;
  }
  err = launch_pdl(attention_prompt_kernel<D, BN, NQ, CTAS>, dim3((unsigned)(plan.ctas * CTAS)),
                   dim3(kPromptThreads), S::kSmem, stream, p, CTAS);
  if (err != cudaSuccess || plan.splits == 1) return err;
  return launch_pdl(attention_prompt_sum_kernel<D, BN, NQ, CTAS>, dim3((unsigned)plan.items, S::kRows * D / 1024), dim3(256),
                    0, stream, p);
}

}  // namespace

// On pairs where sequences may have more rows than one SM takes.
cudaError_t launch_attention_prompt(const AttentionParams& p, int D, void* workspace, cudaStream_t stream) {
  if (D == 64) return launch_with<64, 128, 2, 1>(p, workspace, stream);
  if (D == 128) return launch_with<128, 128, 2, 1>(p, workspace, stream);
  return p.most_columns > 128 ? launch_with<256, 128, 1, 2>(p, workspace, stream)
                              : launch_with<256, 64, 1, 1>(p, workspace, stream);
}

int64_t attention_prompt_workspace(const AttentionParams& p, int D) {
  if (D == 64) return plan_with<64, 128, 2, 1>(p).bytes;
  if (D == 128) return plan_with<128, 128, 2, 1>(p).bytes;
  return p.most_columns > 128 ? plan_with<256, 128, 1, 2>(p).bytes : plan_with<256, 64, 1, 1>(p).bytes;
}

cudaError_t prompt_wait_timeouts(int reset, int* out) {
  cudaError_t err = cudaMemcpyFromSymbol(out, g_prompt_timeouts, sizeof(int));
  const int zero = 0;
  if (err == cudaSuccess && reset) err = cudaMemcpyToSymbol(g_prompt_timeouts, &zero, sizeof(int));
  return err;
}

}  // namespace nvfp4
