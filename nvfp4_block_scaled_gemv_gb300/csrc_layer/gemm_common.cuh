// What the product kernels share: parameters, tiles, and the epilogue.
#pragma once
#include <cstdint>

#include "epilogue.cuh"
#include "layer.h"
#include "quantize.cuh"
#include "tc_ptx.cuh"

namespace nvfp4 {
namespace gemm {

constexpr uint32_t kABytes = 128 * 128;   // 128 rows x 256 elements
constexpr uint32_t kAtoms = 4 * 512;      // a stage's scale atoms of 128 rows
constexpr int kTransposePitch = 33;       // floats between columns of a warp's transpose buffer
constexpr int kUnit = 16;                 // columns an epilogue warp takes at once
constexpr uint32_t kTransposeBytes = kUnit * kTransposePitch * 4;  // per epilogue warp

// Staging of c, per four epilogue warps: buffers of a unit's columns, 128 rows each (two
// of 32-bit values, four of 16-bit ones).
constexpr uint32_t kStageBytesC = 2 * kUnit * 128 * 4;

// An SM's 512 columns of tensor memory are never asked for beyond their number: with
// clusters on both sides, each could hold on one SM what the other waits for on a second, and
// neither that wait (tcgen05.alloc) nor a cluster barrier gives up.  Within a stream the wait
// for the preceding kernels comes before the allocation; between streams shared memory decides
// which CTAs share an SM (it has 228 KB, 1 KB of it reserved per CTA).  A product that takes
// 512 columns asks for enough that no CTA of the tensor-core GEMV fits beside it; one that takes
// 256 leaves room for 256 of theirs at most.  (190 KB for all of them made 53 tokens through 8
// of 64 experts 125 us, 120 with this rule.)
constexpr uint32_t kSmSmem = 228 * 1024, kCtaReserve = 1024;
// What a tensor-core GEMV's CTA needs at least, with its columns: stages of an A tile (128 x
// 128 bytes), a B tile (16 x 128) and eight scale atoms, and 2 KB beside them.
constexpr uint32_t gemv_smem(int stages) { return (uint32_t)stages * (128 * 128 + 16 * 128 + 8 * 512) + 2048; }
constexpr uint32_t gemv_columns(int stages) { return stages == 2 ? 128 : 256; }
// The columns that can be asked for on an SM with a product of this footprint, at most.
constexpr uint32_t most_columns(uint32_t smem, uint32_t columns, uint32_t sm_smem = kSmSmem,
                                uint32_t reserve = kCtaReserve) {
  uint32_t most = columns;
  for (uint32_t n2 = 0; n2 <= 4; ++n2)
    for (uint32_t n4 = 0; n4 <= 2; ++n4)
      for (uint32_t more = 0; more <= 1; ++more) {  // (another product, taken as no larger)
        const uint32_t bytes = (1 + more) * (smem + reserve) + n2 * (gemv_smem(2) + reserve) + n4 * (gemv_smem(4) + reserve);
        const uint32_t all = (1 + more) * columns + n2 * gemv_columns(2) + n4 * gemv_columns(4);
        if (bytes <= sm_smem && all > most) most = all;
      }
  return most;
}
constexpr uint32_t kAloneSmem = 183 * 1024;  // for products of 512 columns, at least

enum Epilogue { kStore = 0, kGatedQuantize = 1 };

struct GemmParams {
  CUtensorMap tmap_a;    // uint8 {K/2, M, G}, box {128, 128, 1}, 128-byte swizzle
  CUtensorMap tmap_b;    // uint8 {K/2, N, L}, box {128, rows, 1}, 128-byte swizzle
  CUtensorMap tmap_sfa;  // pair kernel: the atoms as uint64 {rest_k * 64, G * rest_m}, box {256, 1}
  CUtensorMap tmap_sfb;  // pair kernel: {rest_k * 64, L * rest_n}, box {256, 2}
  CUtensorMap tmap_c;    // c as {M, rows, L}, box {128, kUnit, 1} (if bulk)
  const uint8_t* sfa;    // [G][rest_m][rest_k][512]
  const uint8_t* sfb;    // [L][rest_n][rest_k][512]
  const int4* tiles;     // grouped: {expert, first row, rows, 0}
  const int32_t* tile_count;
  void* c;
  const float* bias;
  const float* alphas;
  uint8_t* q;
  uint8_t* qsf;
  int64_t M, N, c_stride;
  int64_t q_stride, q_atom_row;  // bytes of a row of q, and of an atom row of qsf
  float alpha, encode;
  int32_t c_dtype, activation;
  int32_t paired;        // c takes stores of two adjacent elements
  int32_t bulk;          // c's rows start on 16 bytes: c is stored by TMA
  int32_t rest_m, rest_n, rest_k, kstages;
  int32_t tiles_m;       // tiles of A per group
  int32_t tiles_n;       // dense: N tiles per batch
  int32_t total;         // dense: tiles
  int64_t rows;          // dense: rows of c in all batches
  int32_t c_tile_rows;   // grouped: 0, or the rows of a tile if c's tiles follow each other
};

// One output tile: the mt-th tile of group g's A against rows n0..n0+rows-1 of b.
struct Tile {
  int32_t g;     // batch or expert
  int32_t mt;
  int64_t n0;    // first row of b (within the batch)
  int32_t rows;
};

template <int BN, bool GROUPED>
__device__ __forceinline__ Tile tile_at(const GemmParams& p, int32_t t) {
  Tile o;
  const int32_t nt = t / p.tiles_m;
  o.mt = t - nt * p.tiles_m;
  if constexpr (GROUPED) {
    const int4 e = p.tiles[nt];
    o.g = e.x;
    o.n0 = e.y;
    o.rows = e.z;
  } else {
    o.g = nt / p.tiles_n;
    o.n0 = (int64_t)(nt - o.g * p.tiles_n) * BN;
    o.rows = (int32_t)(p.N - o.n0 < BN ? p.N - o.n0 : BN);
  }
  return o;
}

// True on one lane of a converged warp.  The tcgen05 instructions take their
// descriptors from uniform registers: issued by an elected lane inside control
// flow that the whole warp follows they are one instruction each, while under a
// `lane == 0` branch a 256-row stage's 17 instructions took ~1500 cycles of the
// issuing thread, 4 times the MMAs' own time.
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(is));
  return is != 0;
}

__device__ __forceinline__ uint32_t pack2(__half, float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(__nv_bfloat16, float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float round_to(float, float v) { return v; }
__device__ __forceinline__ __half round_to(__half, float v) { return __float2half_rn(v); }
__device__ __forceinline__ __nv_bfloat16 round_to(__nv_bfloat16, float v) { return __float2bfloat16_rn(v); }

// Columns i and i+1 of this lane's row (a, b), turned with the neighbouring
// lane's into two adjacent rows of one column: column i on even lanes, i+1 on
// odd ones.
template <typename T>
struct Turned;
template <typename T>
struct Turned16 {
  using Store = uint32_t;
  static __device__ __forceinline__ Store turn(float a, float b, bool odd) {
    const uint32_t own = pack2(T(), a, b);
    const uint32_t got = __shfl_xor_sync(0xffffffffu, own, 1);
    return __byte_perm(own, got, odd ? 0x3276 : 0x5410);
  }
};
template <>
struct Turned<__half> : Turned16<__half> {};
template <>
struct Turned<__nv_bfloat16> : Turned16<__nv_bfloat16> {};
template <>
struct Turned<float> {
  using Store = float2;
  static __device__ __forceinline__ Store turn(float a, float b, bool odd) {
    const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
    return make_float2(odd ? got : a, odd ? b : got);
  }
};

// y / (1 + exp(-x)) to (16 + |x| / 4) 2^-24 of itself and 2^-119: the hardware's base-2
// exponential of x log2(e), whose product's rounding is put back (the constant's is not: the
// |x| / 4), and its fast division, which gives 0 for divisors above 2^126.
__device__ __forceinline__ float times_sigmoid(float y, float x) {
  constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
  const float t = -x * kLog2e;
  const float rest = fmaf(-x, kLog2e, -t);  // exact (not finite where t is not)
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  // (beyond, e is 0 or may be infinite already: large x give y, large -x give 0)
  if (fabsf(t) < 127.f) e = fmaf(e, rest * kLn2, e);
  return __fdividef(y, 1.0f + e);
}

// act(y) as in epilogue.cuh, in line for the activations whose instructions matter
// here (the ones made of a sigmoid, in terms of it).
template <int ACT>
__device__ __forceinline__ float activate_inline(float y) {
  if constexpr (ACT == 1) return y > 0.f ? y : (y != y ? y : 0.f);
  if constexpr (ACT == 2) return times_sigmoid(y, y);
  // GELU, tanh form: 1 + tanh(u) = 2 / (1 + exp(-2u))
  if constexpr (ACT == 3) return times_sigmoid(y, 1.5957691216057308f * fmaf(0.044715f * y, y * y, y));
  if constexpr (ACT == 4) return activate(y, 4);
  return y;
}

template <int A>
struct Act {
  static constexpr int value = A;
};

// Columns 0..15 at a TMEM address, without waiting for them.
__device__ __forceinline__ void tmem_load_16(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]),
        "=f"(v[15])
      : "r"(taddr));
}
// Wait for the loads; v is theirs (so that nothing uses it before).
__device__ __forceinline__ void tmem_wait(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]),
                 "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]),
                 "+f"(v[14]), "+f"(v[15])::"memory");
}

// A warp's place in a tile: lane i has the row m of A, all lanes the same
// columns (rows of b).
struct Place {
  int64_t m, row0;   // row of A; row of c or q of the tile's column 0
  int32_t rows;      // columns of the tile
  bool whole;        // all rows of the warp are below M
  float alpha, bias;
  // c by TMA: the four warps' staging (shared address), which buffer is next, their
  // barrier, this warp's quarter, and the tile's place in the map
  uint32_t staging;
  int buffer, barrier, quarter;
  int m0, n0, batch;
  // quantised output: where column 0's codes (of this lane's 8 outputs) and scale go
  // (null past the last block or atom column), and the warp's transpose buffer
  uint8_t* q_at;
  uint8_t* sf_at;
  float* transpose;
};

// Columns n..n+kUnit-1 of the lanes' rows: column i goes to c[(row0 + n + i) * stride + m].
// Neighbouring lanes swap values, so that each stores two adjacent elements of
// one column: half the store instructions.
template <typename T>
__device__ __forceinline__ void store_columns(const GemmParams& p, const Place& w, int n,
                                              const float (&v)[kUnit]) {
  T* at = static_cast<T*>(p.c) + (w.row0 + n) * p.c_stride;
  if (p.paired) {
    const bool odd = (threadIdx.x & 1) != 0;  // (m is the lane plus a multiple of 32)
    at += (odd ? p.c_stride : 0) + (w.m & ~int64_t(1));
    const int64_t step = 2 * p.c_stride;
    if (w.whole && n + kUnit <= w.rows) {  // the same for the whole warp
#pragma unroll
      for (int i = 0; i < kUnit; i += 2) {
        *reinterpret_cast<typename Turned<T>::Store*>(at) = Turned<T>::turn(v[i], v[i + 1], odd);
        at += step;
      }
    } else {
      const int left = w.m < p.M ? w.rows - n - (odd ? 1 : 0) : 0;
#pragma unroll
      for (int i = 0; i < kUnit; i += 2) {
        const typename Turned<T>::Store two = Turned<T>::turn(v[i], v[i + 1], odd);
        if (i < left) *reinterpret_cast<typename Turned<T>::Store*>(at) = two;
        at += step;
      }
    }
  } else if (w.m < p.M) {
    at += w.m;
#pragma unroll
    for (int i = 0; i < kUnit; ++i) {
      if (n + i < w.rows) *at = round_to(T(), v[i]);
      at += p.c_stride;
    }
  }
}

// Whether ok holds for all four warps at a barrier.  (They go on to meet at it for each
// unit, so one that gave up waiting must not leave the others there.)
__device__ __forceinline__ bool four_warps_all(int barrier, bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbar.red.and.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(barrier), "r"((uint32_t)ok)
      : "memory");
  return all != 0;
}

// All but the last N of this thread's bulk stores have read their shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
// They are all complete.
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Columns n..n+kUnit-1 through shared memory: the four warps lay their rows side by
// side and one lane stores the 128 x kUnit box.  One barrier per unit: before it, that
// lane has seen that the store from the buffer of the next unit has been read.  Rows of c past the
// batch's last are not written; a grouped tile's last box may write rows that hold no
// choice.  (A bulk copy per column in place of the box took three times as long as
// the plain stores, ~85 cycles each.)
template <typename T>
__device__ __forceinline__ void bulk_columns(const GemmParams& p, Place& w, int n, const float (&v)[kUnit]) {
  const int lane = threadIdx.x & 31;
  constexpr uint32_t kBytes = kUnit * 128 * (uint32_t)sizeof(T);
  constexpr int kBuffers = (int)(kStageBytesC / kBytes);
  const uint32_t buffer = w.staging + (uint32_t)w.buffer * kBytes;
  w.buffer = w.buffer + 1 == kBuffers ? 0 : w.buffer + 1;
  const uint32_t at = buffer + (uint32_t)sizeof(T) * (uint32_t)(32 * w.quarter + lane);
#pragma unroll
  for (int i = 0; i < kUnit; i += 2) {
    if constexpr (sizeof(T) == 4) {
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + 512u * i), "f"(v[i]) : "memory");
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + 512u * (i + 1)), "f"(v[i + 1]) : "memory");
    } else {
      asm volatile(
          "{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tst.shared.b16 [%0], lo;\n\t"
          "st.shared.b16 [%1], hi;\n\t}" ::"r"(at + 256u * i),
          "r"(at + 256u * (i + 1)), "r"(pack2(T(), v[i], v[i + 1]))
          : "memory");
    }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  const bool sends = w.quarter == 0 && lane == 0;
  if (sends) bulk_wait_read<kBuffers - 2>();
  __syncwarp();
  named_barrier_sync(w.barrier, 128);
  if (sends) {
    if (w.m0 < p.M)
      asm volatile(
          "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(&p.tmap_c),
          "r"(w.m0), "r"(w.n0 + n), "r"(w.batch), "r"(buffer)
          : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
  __syncwarp();
}

// The epilogue of U units of columns, starting at n[u], of a warp's 32 rows (sums v).
// What depends on the call (activation, type) is asked once for all of them: asked
// for each 16 columns, the branches took longer than the columns' own instructions
// (8192 x 8192, K 2048: 60 us, and 47 without any epilogue).
template <int U, bool BULK>
__device__ __forceinline__ void finish_store(const GemmParams& p, Place& w, const int (&n)[U],
                                             float (&v)[U][kUnit]) {
  const uint64_t alpha2 = pack_f32x2(w.alpha, w.alpha), bias2 = pack_f32x2(w.bias, w.bias);
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < kUnit; i += 2) {
      const float2 y = unpack_f32x2(fma2(pack_f32x2(v[u][i], v[u][i + 1]), alpha2, bias2));
      v[u][i] = y.x;
      v[u][i + 1] = y.y;
    }
  if (p.activation != 0) {
    auto each = [&](auto act) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < kUnit; ++i) v[u][i] = activate_inline<decltype(act)::value>(v[u][i]);
    };
    if (p.activation == 2) each(Act<2>());
    if (p.activation == 3) each(Act<3>());
    if (p.activation == 1) each(Act<1>());
    if (p.activation == 4) each(Act<4>());
  }
  auto store = [&](auto type) {
    if constexpr (BULK) {
      if (p.bulk) {
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (n[u] < w.rows) bulk_columns<decltype(type)>(p, w, n[u], v[u]);
        return;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (n[u] < w.rows) store_columns<decltype(type)>(p, w, n[u], v[u]);
  };
  if (p.c_dtype == kBF16)
    store(__nv_bfloat16());
  else if (p.c_dtype == kF16)
    store(__half());
  else
    store(float());
}

// The quantising epilogue of columns n..n+kUnit-1.  The warp's 32 rows are gate and
// input of 16 outputs: one scale block.  Transposed through shared memory, two lanes
// take a column, 8 outputs each.
template <int ACT>
__device__ __forceinline__ void finish_quantize(const GemmParams& p, const Place& w, int n,
                                                const float (&v)[kUnit]) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kUnit; ++i) w.transpose[i * kTransposePitch + lane] = v[i];
  __syncwarp();
  const int col = lane >> 1, half = lane & 1;
  uint64_t h[4];
  float amax = 0.f;
  const float* const mine = w.transpose + col * kTransposePitch + half * 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x =
        activate_inline<ACT>(mine[4 * i] * w.alpha) * (mine[4 * i + 1] * w.alpha) * p.encode;
    const float y =
        activate_inline<ACT>(mine[4 * i + 2] * w.alpha) * (mine[4 * i + 3] * w.alpha) * p.encode;
    amax = abs_max(amax, x, y);
    h[i] = pack_f32x2(x, y);
  }
  amax = abs_max(amax, __shfl_xor_sync(0xffffffffu, amax, 1), 0.f);  // (none is negative)
  uint32_t code = 0x7Fu, q = 0;
  if (is_finite_max(amax)) {
    float s;
    code = block_scale_code(amax, s);
    if (s > 0.f) {
      const float r = scale_reciprocal(s);
      q = quantize_8(h, pack_f32x2(-s, -s), pack_f32x2(r, r));
    }
  }
  const int c = n + col;
  if (c < w.rows) {
    if (w.q_at != nullptr)
      *reinterpret_cast<uint32_t*>(w.q_at + c * p.q_stride) = q;
    else
      code = 0;  // (blocks past the last one pad the last atom column with zero scales)
    // (a tile starts on an atom)
    if (half == 0 && w.sf_at != nullptr)
      w.sf_at[(c >> 7) * p.q_atom_row + (c & 31) * 16 + ((c >> 5) & 3) * 4] = (uint8_t)code;
  }
}

// finish_store or finish_quantize of U units.  BULK: the kernel has staging for c.
template <int EPI, int U, bool BULK>
__device__ __forceinline__ void finish_columns(const GemmParams& p, Place& w, const int (&n)[U],
                                               float (&v)[U][kUnit]) {
  if constexpr (EPI == kStore) {
    finish_store<U, BULK>(p, w, n, v);
  } else {
    auto each = [&](auto act) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (n[u] < w.rows) finish_quantize<decltype(act)::value>(p, w, n[u], v[u]);
    };
    if (p.activation == 2)
      each(Act<2>());
    else if (p.activation == 3)
      each(Act<3>());
    else if (p.activation == 1)
      each(Act<1>());
    else if (p.activation == 4)
      each(Act<4>());
    else
      each(Act<0>());
  }
}

template <int EPI, bool GROUPED>
__device__ __forceinline__ void place_at(Place& w, const GemmParams& p, const Tile& t, int64_t row_tile,
                                         int quarter) {
  w.m = row_tile * 128 + 32 * quarter + (int)(threadIdx.x & 31);
  w.row0 = (GROUPED ? 0 : (int64_t)t.g * p.N) + t.n0;
  if (GROUPED && EPI == kStore && p.c_tile_rows != 0) w.row0 = (t.n0 >> 7) * p.c_tile_rows;
  w.rows = t.rows;
  w.whole = row_tile * 128 + 32 * quarter + 32 <= p.M;
  if constexpr (EPI == kGatedQuantize) {
    const int64_t block = row_tile * 4 + quarter, rest = (p.M + 127) / 128;  // atom columns of M/2
    const int half = threadIdx.x & 1;
    w.q_at = block < p.M / 32 ? p.q + w.row0 * p.q_stride + block * 8 + 4 * half : nullptr;
    w.sf_at = block < 4 * rest ? p.qsf + atom_offset(w.row0, block, rest) : nullptr;
  }
  w.alpha = p.alphas ? p.alphas[t.g] : p.alpha;
  w.bias = EPI == kStore && p.bias && w.m < p.M ? p.bias[(int64_t)t.g * p.M + w.m] : 0.f;
  w.quarter = quarter;
  w.m0 = (int)(row_tile * 128);
  w.n0 = (int)t.n0;
  w.batch = GROUPED ? 0 : t.g;
}

}  // namespace gemm


// The pair kernel (gemm_pair.cu); p complete but for its tensor maps' boxes.
cudaError_t launch_gemm_pair(const gemm::GemmParams& p, int epi, bool grouped, int64_t max_tiles, int sms,
                             cudaStream_t stream);
cudaError_t gemm_pair_wait_timeouts(int reset, int* out);
Footprint pair_footprint(int epi);

}  // namespace nvfp4
