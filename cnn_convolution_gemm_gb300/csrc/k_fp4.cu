// Microscaled 4-bit quantisation, its inverse, and the packing of row-by-row scales.
#include <cuda_runtime.h>

#include "fp4.cuh"
#include "internal.h"

namespace {
using namespace gb::fp4;

constexpr int THREADS = 256;

// One warp per 256 columns of a row: 8 elements a lane, the block's largest
// magnitude by shuffles, codes stored as 4 bytes a lane (128 a warp).
template <int FMT, typename T>
__global__ void __launch_bounds__(THREADS)
    quantize_kernel(const T* __restrict__ x, long long ldx, int rows, int cols, int vec,
                    const TensorScale ts, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const int chunks = (cols + 255) / 256;
  const long long tasks = (long long)rows * chunks;
  const long long step = (long long)gridDim.x * (THREADS / 32);
  for (long long t = (long long)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5); t < tasks;
       t += step) {
    const long long r = t / chunks;
    const int c0 = (int)(t - r * chunks) * 256;
    float v[8];
    load8(x + r * ldx, c0 + (threadIdx.x & 31) * 8, cols, vec, v);
    store_warp_row<FMT>(v, ts, r, c0, cols, codes, scales);
  }
}

template <int FMT, typename T>
__global__ void __launch_bounds__(THREADS)
    dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                      int rows, int cols, int vec, float tensor_scale, T* __restrict__ y,
                      long long ldy) {
  const int chunks = (cols + 255) / 256;
  const long long tasks = (long long)rows * chunks;
  const long long step = (long long)gridDim.x * (THREADS / 32);
  const long long pitch = code_pitch(cols);
  const int tiles = tiles_per_row(FMT, cols);
  for (long long t = (long long)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5); t < tasks;
       t += step) {
    const long long r = t / chunks;
    const int c = (int)(t - r * chunks) * 256 + (threadIdx.x & 31) * 8;
    if (c >= cols) continue;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + r * pitch + c / 2);
    const int b = c / kBlock<FMT>;
    const float s =
        scale_value<FMT>(scales[scale_word_offset(r, b >> 2, tiles) + (b & 3)], tensor_scale);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.5f * e2m1_twice((w >> (4 * i)) & 15u) * s;
    store8(y + r * ldy, c, cols, vec, v);
  }
}

template <int FMT>
__global__ void __launch_bounds__(THREADS)
    pack_scales_kernel(const uint8_t* __restrict__ src, int rows, int cols,
                       uint8_t* __restrict__ scales) {
  const int blocks = (cols + kBlock<FMT> - 1) / kBlock<FMT>;
  const int tiles = tiles_per_row(FMT, cols);
  const long long words = (long long)rows * tiles;
  for (long long i = (long long)blockIdx.x * THREADS + threadIdx.x; i < words;
       i += (long long)gridDim.x * THREADS) {
    const long long r = i / tiles;
    const int tj = (int)(i - r * tiles);
    uint32_t w = 0;
    for (int k = 0; k < 4; ++k)
      if (tj * 4 + k < blocks) w |= (uint32_t)src[r * blocks + tj * 4 + k] << (8 * k);
    *reinterpret_cast<uint32_t*>(scales + scale_word_offset(r, tj, tiles)) = w;
  }
}

int grid_for(long long blocks) {
  const long long most = (long long)gb_num_sms() * 8;
  return (int)(blocks < most ? blocks : most);
}

template <int FMT, typename T>
cudaError_t quantize_t(int rows, int cols, const void* x, long long ldx, float ts, void* codes,
                       void* scales, cudaStream_t st) {
  const long long tasks = (long long)rows * ((cols + 255) / 256);
  quantize_kernel<FMT, T><<<grid_for(gb_ceil_div_ll(tasks, THREADS / 32)), THREADS, 0, st>>>(
      static_cast<const T*>(x), ldx, rows, cols, rows_vec<T>(x, ldx), tensor_scale(ts),
      static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales));
  gb_count_launch();
  return cudaGetLastError();
}

template <int FMT, typename T>
cudaError_t dequantize_t(int rows, int cols, const void* codes, const void* scales, float ts,
                         void* y, long long ldy, cudaStream_t st) {
  const long long tasks = (long long)rows * ((cols + 255) / 256);
  dequantize_kernel<FMT, T><<<grid_for(gb_ceil_div_ll(tasks, THREADS / 32)), THREADS, 0, st>>>(
      static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), rows, cols,
      rows_vec<T>(y, ldy), ts, static_cast<T*>(y), ldy);
  gb_count_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp4_quantize(int fmt, int dtype, int rows, int cols, const void* x,
                                long long ldx, float ts, void* codes, void* scales,
                                cudaStream_t st) {
  if (fmt == CONV_FP4_MX)
    return dtype == CONV_BF16
               ? quantize_t<CONV_FP4_MX, __nv_bfloat16>(rows, cols, x, ldx, ts, codes, scales, st)
               : quantize_t<CONV_FP4_MX, float>(rows, cols, x, ldx, ts, codes, scales, st);
  return dtype == CONV_BF16
             ? quantize_t<CONV_FP4_NV, __nv_bfloat16>(rows, cols, x, ldx, ts, codes, scales, st)
             : quantize_t<CONV_FP4_NV, float>(rows, cols, x, ldx, ts, codes, scales, st);
}

cudaError_t launch_fp4_dequantize(int fmt, int dtype, int rows, int cols, const void* codes,
                                  const void* scales, float ts, void* y, long long ldy,
                                  cudaStream_t st) {
  if (fmt == CONV_FP4_MX)
    return dtype == CONV_BF16
               ? dequantize_t<CONV_FP4_MX, __nv_bfloat16>(rows, cols, codes, scales, ts, y, ldy, st)
               : dequantize_t<CONV_FP4_MX, float>(rows, cols, codes, scales, ts, y, ldy, st);
  return dtype == CONV_BF16
             ? dequantize_t<CONV_FP4_NV, __nv_bfloat16>(rows, cols, codes, scales, ts, y, ldy, st)
             : dequantize_t<CONV_FP4_NV, float>(rows, cols, codes, scales, ts, y, ldy, st);
}

cudaError_t launch_fp4_pack_scales(int fmt, int rows, int cols, const void* src, void* scales,
                                   cudaStream_t st) {
  const long long words = (long long)rows * tiles_per_row(fmt, cols);
  const int grid = grid_for(gb_ceil_div_ll(words, THREADS));
  if (fmt == CONV_FP4_MX)
    pack_scales_kernel<CONV_FP4_MX><<<grid, THREADS, 0, st>>>(
        static_cast<const uint8_t*>(src), rows, cols, static_cast<uint8_t*>(scales));
  else
    pack_scales_kernel<CONV_FP4_NV><<<grid, THREADS, 0, st>>>(
        static_cast<const uint8_t*>(src), rows, cols, static_cast<uint8_t*>(scales));
  gb_count_launch();
  return cudaGetLastError();
}
