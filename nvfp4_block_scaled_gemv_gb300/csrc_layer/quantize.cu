// Quantise and dequantise: rows of 16- or 32-bit values <-> packed E2M1 codes
// with E4M3 block scales (see quantize.cuh for the arithmetic of one block).
//
// Both are one pass over the data, bound by its bytes.  One thread takes one
// 16-element block: 32 or 64 bytes in, 8 bytes of codes and one scale byte out
// (or the other way), so a warp reads and writes whole contiguous lines of a
// row.  In the 128x4-atom layout the threads of the padding (rows up to a
// multiple of 128, blocks up to a multiple of 4) write the zero bytes that the
// product expects there.
#include <cstdint>

#include "layer.h"
#include "ptx.cuh"
#include "quantize.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_float<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// 16 consecutive values, with 16-byte loads (VEC: src 16-byte aligned) or one
// by one.
template <typename T, bool VEC>
__device__ __forceinline__ void load_block(const T* src, float (&y)[16]) {
  if constexpr (VEC) {
    constexpr int kPer = 16 / (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < 16 / kPer; ++i) {
      union {
        uint4 v;
        T t[kPer];
      } u;
      u.v = __ldg(reinterpret_cast<const uint4*>(src) + i);
#pragma unroll
      for (int j = 0; j < kPer; ++j) y[i * kPer + j] = to_float<T>(u.t[j]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = to_float<T>(src[i]);
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_block(T* dst, const float (&y)[16]) {
  if constexpr (VEC) {
    constexpr int kPer = 16 / (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < 16 / kPer; ++i) {
      union {
        uint4 v;
        T t[kPer];
      } u;
#pragma unroll
      for (int j = 0; j < kPer; ++j) u.t[j] = from_float<T>(y[i * kPer + j]);
      reinterpret_cast<uint4*>(dst)[i] = u.v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) dst[i] = from_float<T>(y[i]);
  }
}

template <typename T, bool VEC, bool PERM, bool MAP>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const QuantizeParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t total = p.grid_rows * p.grid_blocks;
  for (int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x; t < total;
       t += (int64_t)gridDim.x * kThreads) {
    const int64_t row = t / p.grid_blocks, kb = t - row * p.grid_blocks;
    // row of the grid -> batch and row in it (padded rows in the atom layout)
    int64_t l = 0, r = row;
    if (PERM && !MAP) {
      l = row / p.rows_pad;
      r = row - l * p.rows_pad;
    }
    const bool real = kb < p.blocks && (MAP || !PERM || r < p.rows);
    uint32_t code = 0;
    uint2 q = make_uint2(0u, 0u);
    if (real) {
      float y[16];
      load_block<T, VEC>(static_cast<const T*>(p.x) + (l * p.rows + r) * p.x_stride + kb * 16, y);
      float amax = 0.f;
      bool finite = true;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        y[i] *= p.encode;
        const float m = fabsf(y[i]);
        finite = finite && m < __int_as_float(0x7f800000);  // false for NaN too
        amax = fmaxf(amax, m);
      }
      if (finite) {
        float s;
        code = block_scale_code(amax, s);
        if (s > 0.f) {
          const float rs = 1.0f / s;
          float lo[8], hi[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            lo[i] = y[i];
            hi[i] = y[8 + i];
          }
          q = make_uint2(quantize_8(lo, s, rs), quantize_8(hi, s, rs));
        }
      } else {
        code = 0x7Fu;
      }
    }
    if constexpr (MAP) {
      for (int j = 0; j < p.copies; ++j) {
        const int64_t dst = p.row_map[r * p.copies + j];
        if (dst < 0 || dst >= p.q_rows) continue;
        if (real) *reinterpret_cast<uint2*>(p.q + dst * p.half_k + kb * 8) = q;
        if constexpr (PERM)
          p.sf[atom_offset(dst, kb, p.rest_k)] = (uint8_t)code;
        else
          p.sf[dst * p.blocks + kb] = (uint8_t)code;
      }
    } else {
      if (real) *reinterpret_cast<uint2*>(p.q + (l * p.rows + r) * p.half_k + kb * 8) = q;
      if constexpr (PERM)
        p.sf[l * (p.rows_pad >> 7) * p.rest_k * 512 + atom_offset(r, kb, p.rest_k)] = (uint8_t)code;
      else
        p.sf[r * p.blocks + kb] = (uint8_t)code;
    }
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const DequantizeParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t total = p.rows * p.L * p.blocks;
  for (int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x; t < total;
       t += (int64_t)gridDim.x * kThreads) {
    const int64_t row = t / p.blocks, kb = t - row * p.blocks;
    uint32_t code;
    if (p.permuted) {
      const int64_t l = row / p.rows, r = row - l * p.rows;
      code = p.sf[l * ((p.rows + 127) / 128) * p.rest_k * 512 + atom_offset(r, kb, p.rest_k)];
    } else {
      code = p.sf[t];
    }
    const uint32_t s2 = e4m3x2_to_f16x2(code);
    const float s = f16_lo_to_f32(s2);
    const uint2 q = *reinterpret_cast<const uint2*>(p.q + row * p.half_k + kb * 8);
    uint32_t h[2][4];
    e2m1x8_to_f16x2x4(q.x, h[0]);
    e2m1x8_to_f16x2x4(q.y, h[1]);
    float y[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[2 * i] = f16_lo_to_f32(h[i / 4][i % 4]) * s * p.scale;  // code * s is exact
      y[2 * i + 1] = f16_hi_to_f32(h[i / 4][i % 4]) * s * p.scale;
    }
    store_block<T, VEC>(static_cast<T*>(p.x) + row * p.x_stride + kb * 16, y);
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

template <typename T>
void (*quantize_for(bool vec, bool perm, bool map))(const QuantizeParams) {
  if (map) {
    if (perm) return vec ? quantize_kernel<T, true, true, true> : quantize_kernel<T, false, true, true>;
    return vec ? quantize_kernel<T, true, false, true> : quantize_kernel<T, false, false, true>;
  }
  if (perm) return vec ? quantize_kernel<T, true, true, false> : quantize_kernel<T, false, true, false>;
  return vec ? quantize_kernel<T, true, false, false> : quantize_kernel<T, false, false, false>;
}

int64_t ctas_for(int64_t threads, int64_t max_ctas) {
  const int64_t n = (threads + kThreads - 1) / kThreads;
  return n < max_ctas ? n : max_ctas;
}

bool rows_aligned_16(const void* x, int64_t stride_bytes) {
  return (reinterpret_cast<uintptr_t>(x) % 16) == 0 && stride_bytes % 16 == 0;
}

}  // namespace

cudaError_t launch_quantize(QuantizeParams p, int dtype, bool permuted, int64_t L, int sms,
                            cudaStream_t stream) {
  const bool map = p.row_map != nullptr;
  p.rows_pad = (p.rows + 127) / 128 * 128;
  p.grid_rows = map ? p.rows : permuted ? L * p.rows_pad : L * p.rows;
  p.grid_blocks = permuted ? 4 * (int64_t)p.rest_k : p.blocks;
  if (!permuted) p.rows = p.grid_rows;  // batches are contiguous rows
  const int64_t size = dtype == kF32 ? 4 : 2;
  const bool vec = rows_aligned_16(p.x, p.x_stride * size);
  auto kern = dtype == kF32    ? quantize_for<float>(vec, permuted, map)
              : dtype == kBF16 ? quantize_for<__nv_bfloat16>(vec, permuted, map)
                               : quantize_for<__half>(vec, permuted, map);
  return launch_pdl(kern, dim3((unsigned)ctas_for(p.grid_rows * p.grid_blocks, (int64_t)sms * 64)),
                    dim3(kThreads), 0, stream, p);
}

cudaError_t launch_fold_signs(const FoldParams& p, int sms, cudaStream_t stream) {
  return launch_pdl(fold_signs_kernel, dim3((unsigned)ctas_for(p.rows * p.L * p.blocks, (int64_t)sms * 64)),
                    dim3(kThreads), 0, stream, p);
}

cudaError_t launch_dequantize(const DequantizeParams& p, int dtype, int sms, cudaStream_t stream) {
  const int64_t size = dtype == kF32 ? 4 : 2;
  const bool vec = rows_aligned_16(p.x, p.x_stride * size);
  auto kern = dtype == kF32    ? (vec ? dequantize_kernel<float, true> : dequantize_kernel<float, false>)
              : dtype == kBF16 ? (vec ? dequantize_kernel<__nv_bfloat16, true>
                                      : dequantize_kernel<__nv_bfloat16, false>)
                               : (vec ? dequantize_kernel<__half, true> : dequantize_kernel<__half, false>);
  return launch_pdl(kern, dim3((unsigned)ctas_for(p.rows * p.L * p.blocks, (int64_t)sms * 64)),
                    dim3(kThreads), 0, stream, p);
}

}  // namespace nvfp4
