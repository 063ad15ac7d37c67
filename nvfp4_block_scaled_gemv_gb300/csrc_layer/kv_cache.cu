// The 4-bit key and value cache: tokens quantised into their slots, and read back
// (see quantize.cuh for the arithmetic of one block, attention.h for the layout).
//
// Both are one pass, bound by the bytes of the 16-bit or 32-bit rows.  A warp takes 8
// tokens and one plane (64 elements) of a head, a lane one 16-element block of K and the
// same one of V, both loads in flight at once.  So it reads 8 pieces of 128 bytes (16-bit
// rows), and, where the tokens' slots follow each other, writes 256 bytes of codes and
// 32 of scales in one run each.
#include <cstdint>

#include "attention.h"
#include "block_io.cuh"
#include "layer.h"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxCtas = 1 << 20;

// A lane's block: its token, head and element, and its place in the cache.
struct Place {
  int64_t token;
  int32_t head, element;
  uint8_t* plane;    // of K in the token's granule, or null: no slot
  int32_t row, block;
};

__device__ __forceinline__ Place place_of(const CacheParams& p, int64_t place) {
  const int lane = threadIdx.x & 31;
  const int per_token = p.heads * p.planes;
  const int64_t group = place / per_token;
  const int rest = (int)(place - group * per_token);
  Place at;
  at.token = group * 8 + (lane >> 2);
  at.head = rest / p.planes;
  const int plane = rest - at.head * p.planes;
  at.block = lane & 3;
  at.element = plane * 64 + at.block * 16;
  at.plane = nullptr;
  at.row = 0;
  if (at.token < p.T) {
    const int64_t slot = __ldg(p.slots + at.token);
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

template <typename T, int ALIGN>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const CacheParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
  for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + warp; i < p.places;
       i += (int64_t)gridDim.x * (kThreads / 32)) {
    const Place at = place_of(p, i);
    if (at.plane == nullptr) continue;
    RawBlock<T> raw[2];
    load_raw<T, ALIGN>(static_cast<const T*>(p.k) + at.token * p.k_token + at.head * p.k_head + at.element, raw[0]);
    load_raw<T, ALIGN>(static_cast<const T*>(p.v) + at.token * p.v_token + at.head * p.v_head + at.element, raw[1]);
    const float encode[2] = {p.encode_k ? __ldg(p.encode_k + at.head) : 1.f,
                             p.encode_v ? __ldg(p.encode_v + at.head) : 1.f};
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint2 q;
      const uint32_t code = quantize_block<T>(raw[s], encode[s], q);
      uint8_t* const plane = at.plane + s * p.planes * kPlaneBytes;
      *reinterpret_cast<uint2*>(plane + at.row * 32 + at.block * 8) = q;
      plane[kPlaneScales + at.row * 4 + at.block] = (uint8_t)code;
    }
  }
}

template <typename T, int ALIGN>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const CacheParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
  for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + warp; i < p.places;
       i += (int64_t)gridDim.x * (kThreads / 32)) {
    const Place at = place_of(p, i);
    if (at.token >= p.T) continue;
    uint2 q[2] = {make_uint2(0u, 0u), make_uint2(0u, 0u)};
    uint32_t code[2] = {0u, 0u};  // (no slot: zeros)
    if (at.plane != nullptr) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint8_t* const plane = at.plane + s * p.planes * kPlaneBytes;
        q[s] = *reinterpret_cast<const uint2*>(plane + at.row * 32 + at.block * 8);
        code[s] = plane[kPlaneScales + at.row * 4 + at.block];
      }
    }
    if (p.k != nullptr)
      dequantize_block<T, ALIGN>(q[0], code[0], p.encode_k ? 1.f / __ldg(p.encode_k + at.head) : 1.f,
                                 static_cast<T*>(p.k) + at.token * p.k_token + at.head * p.k_head + at.element);
    if (p.v != nullptr)
      dequantize_block<T, ALIGN>(q[1], code[1], p.encode_v ? 1.f / __ldg(p.encode_v + at.head) : 1.f,
                                 static_cast<T*>(p.v) + at.token * p.v_token + at.head * p.v_head + at.element);
  }
}

// The widest access (32 or 16 bytes) that every block of every row can take, or 1.
int rows_alignment(const CacheParams& p, int64_t size) {
  const uint64_t bits = (uint64_t)reinterpret_cast<uintptr_t>(p.k) | (uint64_t)reinterpret_cast<uintptr_t>(p.v) |
                        (uint64_t)((p.k_token | p.k_head | p.v_token | p.v_head) * size);
  return bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : 1;
}

template <typename T>
void (*write_for(int align))(const CacheParams) {
  return align == 32 ? kv_write_kernel<T, 32> : align == 16 ? kv_write_kernel<T, 16> : kv_write_kernel<T, 1>;
}
template <typename T>
void (*read_for(int align))(const CacheParams) {
  return align == 32 ? kv_read_kernel<T, 32> : align == 16 ? kv_read_kernel<T, 16> : kv_read_kernel<T, 1>;
}

cudaError_t launch(void (*kern)(const CacheParams), CacheParams& p, cudaStream_t stream) {
  p.places = ((int64_t)p.T + 7) / 8 * p.heads * p.planes;
  const int64_t per_cta = kThreads / 32, need = (p.places + per_cta - 1) / per_cta;
  return launch_pdl(kern, dim3((unsigned)(need < kMaxCtas ? need : kMaxCtas)), dim3(kThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_kv_write(CacheParams p, int dtype, cudaStream_t stream) {
  const int align = rows_alignment(p, dtype == kF32 ? 4 : 2);
  return launch(dtype == kF32    ? write_for<float>(align)
                : dtype == kBF16 ? write_for<__nv_bfloat16>(align)
                                 : write_for<__half>(align),
                p, stream);
}

cudaError_t launch_kv_read(CacheParams p, int dtype, cudaStream_t stream) {
  const int align = rows_alignment(p, dtype == kF32 ? 4 : 2);
  return launch(dtype == kF32    ? read_for<float>(align)
                : dtype == kBF16 ? read_for<__nv_bfloat16>(align)
                                 : read_for<__half>(align),
                p, stream);
}

}  // namespace nvfp4
