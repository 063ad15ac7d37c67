// The 4-bit key and value cache: tokens quantised into their slots, and read back
// (see quantize.cuh for the arithmetic of one block, attention.h for the layout).
//
// Both are one pass, bound by the bytes of the 16-bit or 32-bit rows.  A warp takes 8
// tokens and one plane (64 elements) of a head, or two, a lane one 16-element block of K and the
// same one of V of each plane, all loads in flight at once.  So it reads 8 pieces of 128 bytes a plane
// (16-bit rows), and, where the tokens' slots follow each other, writes 256 bytes of codes and
// 32 of scales in one run each.  16384 tokens x 8 heads of 128 in bf16, writing and reading back together: 29.6 us
// where slots run on within pages, as a prompt's do (86% of the bytes' time at the measured copy's rate), 32.5
// in any order (78%): then a code row is a piece of 32 bytes.  Issue slots are ~58% used (quantising a block is
// ~100 instructions).  24 tokens: 4.3 us, two launches.
#include <cstdint>

#include "attention.h"
#include "block_io.cuh"
#include "layer.h"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxCtas = 1 << 20;

// A lane's block of the first of PLANES planes: its token, head and element, and its place in the
// cache.  The next planes' blocks are 64 elements and kPlaneBytes on.
struct Place {
  int64_t token;
  int32_t head, element;
  uint8_t* plane;    // of K in the token's granule, or null: no slot
  int32_t row, block;
};

template <int PLANES>
__device__ __forceinline__ Place place_of(const CacheParams& p, int64_t place) {
  const int lane = threadIdx.x & 31;
  const int runs = p.planes / PLANES, per_token = p.heads * runs;
  const int64_t group = p.places < (int64_t(1) << 32) ? (int64_t)((uint32_t)place / (uint32_t)per_token) : place / per_token;
  const int rest = (int)(place - group * per_token);
  Place at;
  at.token = group * 8 + (lane >> 2);
  at.head = runs == 1 ? rest : rest / runs;
  const int plane = (rest - at.head * runs) * PLANES;
  at.block = lane & 3;
  at.element = plane * 64 + at.block * 16;
  at.plane = nullptr;
  at.row = 0;
  if (at.token < p.T) {
    const int64_t slot = ld_now(p.slots + at.token);
    if (slot >= 0 && slot < p.capacity) {
      const int64_t page = p.capacity <= 0xffffffffll ? (int64_t)((uint32_t)slot / (uint32_t)p.page_size)
                                                      : slot / p.page_size;
      const int32_t in_page = (int32_t)(slot - page * p.page_size);
      const int64_t granule = (page * p.heads + at.head) * p.granules + in_page / kGranuleTokens;
      at.row = in_page % kGranuleTokens;
      at.plane = p.cache + (granule * 2 * p.planes + plane) * kPlaneBytes;
    }
  }
  return at;
}

template <typename T, int ALIGN, int PLANES>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const CacheParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
  for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + warp; i < p.places;
       i += (int64_t)gridDim.x * (kThreads / 32)) {
    const Place at = place_of<PLANES>(p, i);
    if (at.plane == nullptr) continue;
    const T* const x[2] = {static_cast<const T*>(p.k) + at.token * p.k_token + at.head * p.k_head + at.element,
                           static_cast<const T*>(p.v) + at.token * p.v_token + at.head * p.v_head + at.element};
    RawBlock<T> raw[2][PLANES];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int c = 0; c < PLANES; ++c) load_raw<T, ALIGN>(x[s] + 64 * c, raw[s][c]);
    const float encode[2] = {p.encode_k ? ld_now(p.encode_k + at.head) : 1.f,
                             p.encode_v ? ld_now(p.encode_v + at.head) : 1.f};
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint8_t* const to = at.plane + s * p.planes * kPlaneBytes + at.row * 32 + at.block * 8;
      uint8_t* const scale_to = at.plane + s * p.planes * kPlaneBytes + kPlaneScales + at.row * 4 + at.block;
#pragma unroll
      for (int c = 0; c < PLANES; ++c) {
        uint2 q;
        const uint32_t code = quantize_block<T>(raw[s][c], encode[s], q);
        *reinterpret_cast<uint2*>(to + c * kPlaneBytes) = q;
        scale_to[c * kPlaneBytes] = (uint8_t)code;
      }
    }
  }
}

template <typename T, int ALIGN, int PLANES>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const CacheParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
  for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + warp; i < p.places;
       i += (int64_t)gridDim.x * (kThreads / 32)) {
    const Place at = place_of<PLANES>(p, i);
    if (at.token >= p.T) continue;
    uint2 q[2][PLANES];
    uint32_t code[2][PLANES];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int c = 0; c < PLANES; ++c) q[s][c] = make_uint2(0u, 0u), code[s][c] = 0u;  // (no slot: zeros)
    if (at.plane != nullptr) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint8_t* const from = at.plane + s * p.planes * kPlaneBytes + at.row * 32 + at.block * 8;
        const uint8_t* const scale_at = at.plane + s * p.planes * kPlaneBytes + kPlaneScales + at.row * 4 + at.block;
#pragma unroll
        for (int c = 0; c < PLANES; ++c) {
          q[s][c] = *reinterpret_cast<const uint2*>(from + c * kPlaneBytes);
          code[s][c] = scale_at[c * kPlaneBytes];
        }
      }
    }
    if (p.k != nullptr) {
      const float decode = p.encode_k ? __frcp_rn(ld_now(p.encode_k + at.head)) : 1.f;
      T* const to = static_cast<T*>(p.k) + at.token * p.k_token + at.head * p.k_head + at.element;
#pragma unroll
      for (int c = 0; c < PLANES; ++c) dequantize_block<T, ALIGN>(q[0][c], code[0][c], decode, to + 64 * c);
    }
    if (p.v != nullptr) {
      const float decode = p.encode_v ? __frcp_rn(ld_now(p.encode_v + at.head)) : 1.f;
      T* const to = static_cast<T*>(p.v) + at.token * p.v_token + at.head * p.v_head + at.element;
#pragma unroll
      for (int c = 0; c < PLANES; ++c) dequantize_block<T, ALIGN>(q[1][c], code[1][c], decode, to + 64 * c);
    }
  }
}

// The widest access (32 or 16 bytes) that every block of every row can take, or 1.
int rows_alignment(const CacheParams& p, int64_t size) {
  const uint64_t bits = (uint64_t)reinterpret_cast<uintptr_t>(p.k) | (uint64_t)reinterpret_cast<uintptr_t>(p.v) |
                        (uint64_t)((p.k_token | p.k_head | p.v_token | p.v_head) * size);
  return bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : 1;
}

// Two planes a lane share the work on its place, where heads have more than one and every row's
// loads are the widest (and there are enough of them for every SM all the same).
int planes_at_once(const CacheParams& p, int align) {
  return p.planes > 1 && align == 32 && (int64_t)p.T * p.heads * p.planes >= 32768 ? 2 : 1;
}
template <typename T>
void (*write_for(int align, int planes))(const CacheParams) {
  if (planes == 2) return kv_write_kernel<T, 32, 2>;
  return align == 32 ? kv_write_kernel<T, 32, 1> : align == 16 ? kv_write_kernel<T, 16, 1> : kv_write_kernel<T, 1, 1>;
}
template <typename T>
void (*read_for(int align, int planes))(const CacheParams) {
  if (planes == 2) return kv_read_kernel<T, 32, 2>;
  return align == 32 ? kv_read_kernel<T, 32, 1> : align == 16 ? kv_read_kernel<T, 16, 1> : kv_read_kernel<T, 1, 1>;
}

cudaError_t launch(void (*kern)(const CacheParams), CacheParams& p, int planes, cudaStream_t stream) {
  p.places = ((int64_t)p.T + 7) / 8 * p.heads * (p.planes / planes);
  const int64_t per_cta = kThreads / 32, need = (p.places + per_cta - 1) / per_cta;
  return launch_pdl(kern, dim3((unsigned)(need < kMaxCtas ? need : kMaxCtas)), dim3(kThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_kv_write(CacheParams p, int dtype, cudaStream_t stream) {
  const int align = rows_alignment(p, dtype == kF32 ? 4 : 2);
  const int planes = planes_at_once(p, align);
  return launch(dtype == kF32    ? write_for<float>(align, planes)
                : dtype == kBF16 ? write_for<__nv_bfloat16>(align, planes)
                                 : write_for<__half>(align, planes),
                p, planes, stream);
}

cudaError_t launch_kv_read(CacheParams p, int dtype, cudaStream_t stream) {
  const int align = rows_alignment(p, dtype == kF32 ? 4 : 2);
  const int planes = planes_at_once(p, align);
  return launch(dtype == kF32    ? read_for<float>(align, planes)
                : dtype == kBF16 ? read_for<__nv_bfloat16>(align, planes)
                                 : read_for<__half>(align, planes),
                p, planes, stream);
}

}  // namespace nvfp4
