// Quantise and dequantise: rows of 16- or 32-bit values <-> packed E2M1 codes
// with E4M3 block scales (see quantize.cuh for the arithmetic of one block).
//
// Both are one pass over the data, bound by its bytes.  One thread takes one
// 16-element block: 32 or 64 bytes in, 8 bytes of codes and one scale byte out
// (or the other way), so a warp takes 32 consecutive blocks of a row.  A block costs
// the quantise kernel ~130 instructions, close to the time of its bytes, so that a
// warp of large inputs has the loads of 4 blocks in flight before it works on the
// first.  In the 128x4-atom layout the threads of the padding (rows up to a multiple
// of 128, blocks up to a multiple of 4) write the zero bytes that the product
// expects there.  16384 x 8192 bf16 with atoms: 52.0 us, 6.61 TB/s, 97% of the measured
// copy; back 51.2 us, 99%.
#include <cstdint>

#include "block_io.cuh"
#include "layer.h"
#include "ptx.cuh"
#include "quantize.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxCtas = 1 << 20;

enum Target { kPlain = 0, kAtoms = 1, kMapPlain = 2, kMapAtoms = 3 };

// Warps take places (row, 32 U blocks) in the order of memory: the place is worked
// out once and its U loads, U * 1 KB of a 16-bit row, are issued before the first
// block is worked on; with atoms the rows and the blocks count their padding too.
// (A sector of an atom holds 4 blocks of 8 rows, so a warp writes 32 scale bytes as 8
// words.  Taking the 8 rows together, by one warp or by the warps of a CTA, writes
// whole sectors but reads x in 8 streams of rows at once, and was 5-10 us slower at
// 16384 x 8192; a persistent grid ran between 57 and 79 us there by its size, as its
// stride fell on the memory channels.)
template <typename T, int ALIGN, int TARGET, int U>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const QuantizeParams p) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr bool kMap = TARGET >= kMapPlain;
  constexpr bool kIsAtoms = (TARGET & 1) != 0;
  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
  const int32_t width = kIsAtoms ? 4 * p.rest_k : p.blocks;
  for (int64_t place = (int64_t)blockIdx.x * (kThreads / 32) + warp; place < p.places;
       place += (int64_t)gridDim.x * (kThreads / 32)) {
    const int64_t row =
        p.places < (int64_t(1) << 32) ? (int64_t)((uint32_t)place / (uint32_t)p.chunks) : place / p.chunks;
    const int32_t kb0 = (int32_t)(place - row * p.chunks) * (32 * U) + lane;
    int64_t from = row;  // the row of x, or -1 for padding
    if (TARGET == kAtoms) {
      const int64_t l = p.one_batch ? 0 : row / p.rows_pad;
      const int64_t r = row - l * p.rows_pad;
      from = r < p.rows ? l * p.rows + r : -1;
    }
    const T* const x = static_cast<const T*>(p.x) + from * p.x_stride + (int64_t)kb0 * 16;
    RawBlock<T> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (from >= 0 && kb0 + 32 * u < p.blocks) load_raw<T, ALIGN>(x + 512 * u, raw[u]);
    uint2* const q_at = reinterpret_cast<uint2*>(p.q + from * p.half_k) + kb0;
    // (rows_pad is a multiple of 128: the batches' atom rows follow each other)
    uint8_t* const sf_at = p.sf + (kIsAtoms ? atom_offset(row, kb0, p.rest_k) : row * p.blocks + kb0);
    constexpr int kSfStep = kIsAtoms ? 8 * 512 : 32;  // from one 32 blocks to the next
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int32_t kb = kb0 + 32 * u;
      uint2 q = make_uint2(0u, 0u);
      const bool real = from >= 0 && kb < p.blocks;
      const uint32_t code = real ? quantize_block<T>(raw[u], p.encode, q) : 0u;
      if constexpr (kMap) {
        if (kb < width)
          for (int j = 0; j < p.copies; ++j) {
            const int64_t dst = p.row_map[row * p.copies + j];
            if (dst < 0 || dst >= p.q_rows) continue;
            if (real) *(reinterpret_cast<uint2*>(p.q + dst * p.half_k) + kb) = q;
            p.sf[kIsAtoms ? atom_offset(dst, kb, p.rest_k) : dst * p.blocks + kb] = (uint8_t)code;
          }
      } else {
        if (real) q_at[32 * u] = q;
        if (kb < width) sf_at[kSfStep * u] = (uint8_t)code;
      }
    }
  }
}

// The sort of few choices (at most kPlaceMost) and the quantisation of the tokens into
// the experts' rows, in one launch: a CTA per token, which sorts all the choices for
// itself (a count of every expert's, and for its own token's the ones before them)
// instead of waiting for another kernel to have done so.  The first CTA leaves the
// sort's results for the products.
template <typename T, int ALIGN>
__global__ void __launch_bounds__(kThreads) place_kernel(const PlaceParams p) {
  __shared__ int32_t ids[kPlaceMost];
  __shared__ int32_t counts[kMaxExperts], first[kMaxExperts];  // choices; tiles before the expert's
  __shared__ int32_t part[kThreads / 32];
  __shared__ int32_t rows[kMaxTopK];
  pdl_launch_dependents();
  const SortParams& s = p.sort;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = (int)s.n, k = p.quantize.copies;
  for (int e = threadIdx.x; e < s.E; e += kThreads) counts[e] = 0;
  pdl_wait();
  // the first block of x while the sort goes on
  const T* const x = static_cast<const T*>(p.quantize.x) + (int64_t)blockIdx.x * p.quantize.x_stride;
  RawBlock<T> raw;
  if ((int)threadIdx.x < p.quantize.blocks) load_raw<T, ALIGN>(x + 16 * threadIdx.x, raw);
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int32_t e = s.ids[i];
    ids[i] = e >= 0 && e < s.E ? e : -1;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads)
    if (ids[i] >= 0) atomicAdd(&counts[ids[i]], 1);  // (a count: the order does not show)
  __syncthreads();
  // tiles before each expert: every thread has some consecutive experts
  const int per = (s.E + kThreads - 1) / kThreads, e0 = threadIdx.x * per;
  int32_t mine = 0;
  for (int e = e0; e < e0 + per && e < s.E; ++e) mine += (counts[e] + s.tile_rows - 1) / s.tile_rows;
  int32_t upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int32_t o = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == 31) part[warp] = upto;
  __syncthreads();
  for (int w = 0; w < warp; ++w) upto += part[w];
  int32_t at = upto - mine;
  for (int e = e0; e < e0 + per && e < s.E; ++e) {
    first[e] = at;
    at += (counts[e] + s.tile_rows - 1) / s.tile_rows;
  }
  __syncthreads();
  // the rows of this token's choices: a warp counts the ones before
  for (int j = warp; j < k; j += kThreads / 32) {
    const int i = (int)blockIdx.x * k + j;
    const int32_t e = ids[i];
    int32_t before = 0;
    for (int b = lane; b < i; b += 32) before += ids[b] == e ? 1 : 0;
    before = __reduce_add_sync(0xffffffffu, before);
    const int32_t tile = before / s.tile_rows;
    const int32_t row = e < 0 ? -1 : (first[e] + tile) * s.pitch + before - tile * s.tile_rows;
    if (lane == 0) {
      rows[j] = row;
      s.rows[i] = row < 0 ? -1 : row - (row >> 7) * p.skip;
    }
  }
  if (blockIdx.x == 0) {
    if (threadIdx.x == kThreads - 1) *s.tile_count = upto;
    for (int e = threadIdx.x; e < s.E; e += kThreads) {
      s.counts[e] = counts[e];
      s.starts[e] = first[e] * s.pitch;
      for (int i = 0, left = counts[e]; left > 0; ++i, left -= s.tile_rows)
        s.tiles[first[e] + i] = make_int4(e, (first[e] + i) * s.pitch, min(left, s.tile_rows), 0);
    }
  }
  __syncthreads();
  const QuantizeParams& z = p.quantize;
  for (int kb = threadIdx.x; kb < 4 * z.rest_k; kb += kThreads) {
    if (kb >= kThreads && kb < z.blocks) load_raw<T, ALIGN>(x + 16 * kb, raw);
    uint2 q = make_uint2(0u, 0u);
    const uint32_t code = kb < z.blocks ? quantize_block<T>(raw, z.encode, q) : 0u;
    for (int j = 0; j < k; ++j) {
      const int64_t dst = rows[j];
      if (dst < 0) continue;
      if (kb < z.blocks) *(reinterpret_cast<uint2*>(z.q + dst * z.half_k) + kb) = q;
      z.sf[atom_offset(dst, kb, z.rest_k)] = (uint8_t)code;
    }
  }
}

// Places as in quantize_kernel (no padding).
template <typename T, int ALIGN, bool PERM, int U>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const DequantizeParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
  for (int64_t place = (int64_t)blockIdx.x * (kThreads / 32) + warp; place < p.places;
       place += (int64_t)gridDim.x * (kThreads / 32)) {
    const int64_t row =
        p.places < (int64_t(1) << 32) ? (int64_t)((uint32_t)place / (uint32_t)p.chunks) : place / p.chunks;
    const int32_t kb0 = (int32_t)(place - row * p.chunks) * (32 * U) + lane;
    const uint2* const q_at = reinterpret_cast<const uint2*>(p.q + row * p.half_k) + kb0;
    const uint8_t* sf_at = p.sf + row * p.blocks + kb0;
    if constexpr (PERM) {
      const int64_t l = p.L == 1 ? 0 : row / p.rows;
      sf_at = p.sf + l * ((p.rows + 127) / 128) * p.rest_k * 512 + atom_offset(row - l * p.rows, kb0, p.rest_k);
    }
    constexpr int kSfStep = PERM ? 8 * 512 : 32;
    uint2 q[U];
    uint32_t code[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (kb0 + 32 * u < p.blocks) {
        q[u] = ld_now(q_at + 32 * u);
        code[u] = sf_at[kSfStep * u];
      }
    T* const x = static_cast<T*>(p.x) + row * p.x_stride + (int64_t)kb0 * 16;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (kb0 + 32 * u < p.blocks) dequantize_block<T, ALIGN>(q[u], code[u], p.scale, x + 512 * u);
  }
}

// Moves the sign of a scale code into the 16 elements it scales.
__global__ void __launch_bounds__(kThreads) fold_signs_kernel(const FoldParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t total = p.rows * p.L * p.blocks;
  for (int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x; t < total;
       t += (int64_t)gridDim.x * kThreads) {
    const int64_t row = t / p.blocks, kb = t - row * p.blocks;
    const int64_t l = row / p.rows, r = row - l * p.rows;
    uint8_t* const code =
        p.sf + (p.permuted ? l * ((p.rows + 127) / 128) * p.rest_k * 512 + atom_offset(r, kb, p.rest_k) : t);
    const uint8_t c = *code;
    if (c & 0x80u) {
      *code = c & 0x7Fu;
      uint2* const q = reinterpret_cast<uint2*>(p.a + row * p.half_k + kb * 8);
      *q = make_uint2(q->x ^ 0x88888888u, q->y ^ 0x88888888u);
    }
  }
}

template <typename T, int ALIGN, int U>
void (*quantize_with(bool perm, bool map))(const QuantizeParams) {
  if (map) return perm ? quantize_kernel<T, ALIGN, kMapAtoms, U> : quantize_kernel<T, ALIGN, kMapPlain, U>;
  return perm ? quantize_kernel<T, ALIGN, kAtoms, U> : quantize_kernel<T, ALIGN, kPlain, U>;
}
template <typename T>
void (*quantize_for(int align, bool perm, bool map, int u))(const QuantizeParams) {
  constexpr int kMany = sizeof(T) == 4 ? 2 : 4;
  if (align == 32) return u > 1 ? quantize_with<T, 32, kMany>(perm, map) : quantize_with<T, 32, 1>(perm, map);
  return align == 16 ? quantize_with<T, 16, 1>(perm, map) : quantize_with<T, 1, 1>(perm, map);
}

int64_t ctas_for(int64_t threads, int64_t max_ctas) {
  const int64_t n = (threads + kThreads - 1) / kThreads;
  return n < max_ctas ? n : max_ctas;
}

// The widest load (32 or 16 bytes) that every block of every row can take, or 1.
int row_alignment(const void* x, int64_t stride_bytes) {
  const uint64_t bits = (uint64_t)reinterpret_cast<uintptr_t>(x) | (uint64_t)stride_bytes;
  return bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : 1;
}

}  // namespace

cudaError_t launch_quantize(QuantizeParams p, int dtype, bool permuted, int64_t L, int sms,
                            cudaStream_t stream) {
  const bool map = p.row_map != nullptr;
  const int64_t size = dtype == kF32 ? 4 : 2;
  const int align = row_alignment(p.x, p.x_stride * size);
  p.rows_pad = (p.rows + 127) / 128 * 128;
  p.one_batch = L == 1;
  if (!permuted) p.rows *= L;  // the batches' rows follow each other
  const int32_t width = permuted ? 4 * p.rest_k : p.blocks;
  const int64_t rows = permuted && !map ? L * p.rows_pad : p.rows;
  // several blocks per lane when rows are long enough to use them and there are
  // enough to fill the GPU all the same (8 CTAs of 8 warps per SM)
  const int most = dtype == kF32 ? 2 : 4;
  const bool many = align == 32 && width >= 32 * most && rows * (width / (32 * most)) >= (int64_t)sms * 64;
  const int u = many ? most : 1;
  p.chunks = (width + 32 * u - 1) / (32 * u);
  p.places = rows * p.chunks;
  auto kern = dtype == kF32    ? quantize_for<float>(align, permuted, map, u)
              : dtype == kBF16 ? quantize_for<__nv_bfloat16>(align, permuted, map, u)
                               : quantize_for<__half>(align, permuted, map, u);
  const int64_t per_cta = kThreads / 32, need = (p.places + per_cta - 1) / per_cta;
  return launch_pdl(kern, dim3((unsigned)(need < kMaxCtas ? need : kMaxCtas)), dim3(kThreads), 0, stream, p);
}

template <typename T>
void (*place_for(int align))(const PlaceParams) {
  return align == 32 ? place_kernel<T, 32> : align == 16 ? place_kernel<T, 16> : place_kernel<T, 1>;
}

cudaError_t launch_place(const PlaceParams& p, int dtype, int64_t T, cudaStream_t stream) {
  const int align = row_alignment(p.quantize.x, p.quantize.x_stride * 2);
  auto kern = dtype == kBF16 ? place_for<__nv_bfloat16>(align) : place_for<__half>(align);
  return launch_pdl(kern, dim3((unsigned)T), dim3(kThreads), 0, stream, p);
}

cudaError_t launch_fold_signs(const FoldParams& p, int sms, cudaStream_t stream) {
  return launch_pdl(fold_signs_kernel, dim3((unsigned)ctas_for(p.rows * p.L * p.blocks, (int64_t)sms * 64)),
                    dim3(kThreads), 0, stream, p);
}

template <typename T, int ALIGN, int U>
void (*dequantize_with(bool perm))(const DequantizeParams) {
  return perm ? dequantize_kernel<T, ALIGN, true, U> : dequantize_kernel<T, ALIGN, false, U>;
}
template <typename T>
void (*dequantize_for(int align, bool perm, int u))(const DequantizeParams) {
  if (align == 32) return u > 1 ? dequantize_with<T, 32, 4>(perm) : dequantize_with<T, 32, 1>(perm);
  return align == 16 ? dequantize_with<T, 16, 1>(perm) : dequantize_with<T, 1, 1>(perm);
}

cudaError_t launch_dequantize(DequantizeParams p, int dtype, int sms, cudaStream_t stream) {
  const int align = row_alignment(p.x, p.x_stride * (dtype == kF32 ? 4 : 2));
  const int64_t rows = p.rows * p.L;
  const bool many = align == 32 && p.blocks >= 128 && rows * (p.blocks / 128) >= (int64_t)sms * 64;
  const int u = many ? 4 : 1;
  p.chunks = (p.blocks + 32 * u - 1) / (32 * u);
  p.places = rows * p.chunks;
  auto kern = dtype == kF32    ? dequantize_for<float>(align, p.permuted, u)
              : dtype == kBF16 ? dequantize_for<__nv_bfloat16>(align, p.permuted, u)
                               : dequantize_for<__half>(align, p.permuted, u);
  const int64_t per_cta = kThreads / 32, need = (p.places + per_cta - 1) / per_cta;
  return launch_pdl(kern, dim3((unsigned)(need < kMaxCtas ? need : kMaxCtas)), dim3(kThreads), 0, stream, p);
}

}  // namespace nvfp4
