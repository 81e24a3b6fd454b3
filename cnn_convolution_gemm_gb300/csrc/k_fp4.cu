// Microscaled 4-bit quantisation, its inverse, and the packing of row-by-row scales.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "fp4.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace {
using namespace gb::fp4;

constexpr int THREADS = 256;
constexpr int ROWS = 2;  // rows whose loads a warp issues together

// A warp works on 512 columns of a row, 16 to a lane (32 bytes of bf16), and walks over
// rows.  Both directions should move bytes only: the loads of several rows are in flight
// per warp, and the instructions of an element are few.  Rows of up to 256 (128) columns
// share a warp two (four) at a time.  wx (a power of two up to 8) warps of a block lie
// side by side along a row, the others below one another.  Measured: 16384 x 8192 bf16 to
// NV 58 us and back 55 us (5.9 and 6.3 TB/s; bound by HBM), 12544 x 256 to MX 2.7 us.
struct Walk {
  int c;               // the lane's first column
  long long row, step; // the lane's first row, and rows between its rows
};
// NARROW: wx_log2 < 0, 1 << -wx_log2 rows to a warp
template <bool NARROW>
__device__ __forceinline__ Walk walk(int wx_log2) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Walk w;
  if constexpr (NARROW) {
    const int lanes_log2 = 5 + wx_log2;  // lanes of a row
    const int wy = (THREADS / 32) << -wx_log2;
    w.c = (lane & ((1 << lanes_log2) - 1)) * 16;
    w.row = (long long)blockIdx.y * wy + (warp << -wx_log2) + (lane >> lanes_log2);
    w.step = (long long)gridDim.y * wy;
    return w;
  }
  const int wy = (THREADS / 32) >> wx_log2;
  w.c = (((int)blockIdx.x << wx_log2) + (warp & ((1 << wx_log2) - 1))) * 512 +
        (threadIdx.x & 31) * 16;
  w.row = (long long)blockIdx.y * wy + (warp >> wx_log2);
  w.step = (long long)gridDim.y * wy;
  return w;
}

// ANY: rows that 32-byte accesses do not fit
template <int FMT, typename T, bool NARROW, bool ANY>
__global__ void __launch_bounds__(THREADS)
    quantize_kernel(const T* __restrict__ x, long long ldx, int rows, int cols, int wx_log2,
                    const TensorScale ts, uint8_t* __restrict__ codes,
                    uint8_t* __restrict__ scales) {
  gb::allow_dependents();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Walk w = walk<NARROW>(wx_log2);
  if (!NARROW && w.c - (int)(threadIdx.x & 31) * 16 >= cols) return;  // the whole warp
  // the lanes of a warp go round together: the shuffles below are the warp's
  const long long lead = w.row - (NARROW ? (threadIdx.x & 31) >> (5 + wx_log2) : 0);
  for (long long r0 = w.row, l0 = lead; l0 < rows; r0 += ROWS * w.step, l0 += ROWS * w.step) {
    std::conditional_t<ANY, RawAny16<T>, Raw16<T>> raw[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const long long r = r0 + i * w.step;
      if (r >= rows) continue;
      if constexpr (ANY)
        raw[i].load(x + r * ldx, w.c, cols, r == 0, r == rows - 1);
      else
        raw[i].load(x + r * ldx, w.c, cols, true);
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const long long r = r0 + i * w.step;
      if (l0 + i * w.step >= rows) break;
      float v[16];
      raw[i].get(v);
      uint2 packed;
      uint32_t word;
      quantize16<FMT>(v, ts, packed, word);
      if (!NARROW || r < rows) store_quantized16<FMT>(packed, word, r, w.c, cols, codes, scales);
    }
  }
}

template <int FMT, typename T, bool NARROW, bool ANY>
__global__ void __launch_bounds__(THREADS)
    dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                      int rows, int cols, int wx_log2, float tensor_scale,
                      T* __restrict__ y, long long ldy) {
  gb::allow_dependents();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Walk w = walk<NARROW>(wx_log2);
  const int lane = NARROW ? w.c / 16 : (int)(threadIdx.x & 31);  // of the row's in this warp
  // ANY: the lanes of a warp hand elements to one another, and go round together
  if (w.c - (ANY ? lane * 16 : 0) >= cols) return;
  const long long lead =
      w.row - (NARROW && ANY ? (int)(threadIdx.x & 31) >> (5 + wx_log2) : 0);
  const long long pitch = code_pitch(cols);
  const int tiles = tiles_per_row(FMT, cols), b = w.c / kBlock<FMT>;
  for (long long r0 = w.row, l0 = lead; l0 < rows; r0 += ROWS * w.step, l0 += ROWS * w.step) {
    uint2 code[ROWS];
    uint32_t byte[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const long long r = r0 + i * w.step;
      if (r >= rows || w.c >= cols) continue;
      code[i] = *reinterpret_cast<const uint2*>(codes + r * pitch + w.c / 2);
      byte[i] = scales[scale_word_offset(r, b >> 2, tiles) + (b & 3)];
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const long long r = r0 + i * w.step;
      if ((ANY ? l0 + i * w.step : r) >= rows) continue;
      const float s = scale_value<FMT>(byte[i], tensor_scale);
      float lo[8], hi[8], v[16];
      unpack8_e2m1(code[i].x, lo);
      unpack8_e2m1(code[i].y, hi);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[k] = lo[k] * s;
        v[8 + k] = hi[k] * s;
      }
      if constexpr (ANY)
        store_warp_any16(y + r * ldy, w.c - lane * 16, r < rows ? cols : 0, v, lane,
                         NARROW ? 32 >> -wx_log2 : 32);
      else
        store16(y + r * ldy, w.c, cols, v);
    }
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

// Grid of a walk over rows x cols: the columns covered once, as many rows at a time as
// fill the SMs (8 blocks each) with ROWS rows to a warp.
struct Shape {
  dim3 grid;
  int wx_log2;
};
Shape walk_shape(int rows, int cols) {
  Shape s;
  const int chunks = (int)gb_ceil_div_ll(cols, 512);
  s.wx_log2 = cols <= 128 ? -2 : cols <= 256 ? -1 : 0;
  while (s.wx_log2 >= 0 && s.wx_log2 < 3 && (1 << s.wx_log2) < chunks) ++s.wx_log2;
  const int wy = s.wx_log2 < 0 ? (THREADS / 32) << -s.wx_log2 : (THREADS / 32) >> s.wx_log2;
  const int gx = s.wx_log2 < 0 ? 1 : gb_ceil_div(chunks, 1 << s.wx_log2);
  const long long need = gb_ceil_div_ll(rows, ROWS * wy);
  const long long gy = std::min<long long>(need, std::max(1, gb_num_sms() * 8 / gx));
  s.grid = dim3((unsigned)gx, (unsigned)gy);
  return s;
}

// Launch that may set up while the kernel before it drains (it waits for that kernel's
// end before it touches global memory).
template <typename... P, typename... A>
cudaError_t launch_walk(void (*kern)(P...), dim3 grid, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  if (e == cudaSuccess) gb_count_launch();
  return e;
}

template <int FMT, typename T>
cudaError_t quantize_t(int rows, int cols, const void* x, long long ldx, float ts, void* codes,
                       void* scales, cudaStream_t st) {
  const Shape s = walk_shape(rows, cols);
  const bool narrow = s.wx_log2 < 0;
  auto* kern = rows_vec<T>(x, ldx, 32)
                   ? (narrow ? quantize_kernel<FMT, T, true, false>
                             : quantize_kernel<FMT, T, false, false>)
                   : (narrow ? quantize_kernel<FMT, T, true, true>
                             : quantize_kernel<FMT, T, false, true>);
  return launch_walk(kern, s.grid, st, static_cast<const T*>(x), ldx, rows, cols, s.wx_log2,
                     tensor_scale(ts), static_cast<uint8_t*>(codes),
                     static_cast<uint8_t*>(scales));
}

template <int FMT, typename T>
cudaError_t dequantize_t(int rows, int cols, const void* codes, const void* scales, float ts,
                         void* y, long long ldy, cudaStream_t st) {
  const Shape s = walk_shape(rows, cols);
  const bool narrow = s.wx_log2 < 0;
  auto* kern = rows_vec<T>(y, ldy, 32)
                   ? (narrow ? dequantize_kernel<FMT, T, true, false>
                             : dequantize_kernel<FMT, T, false, false>)
                   : (narrow ? dequantize_kernel<FMT, T, true, true>
                             : dequantize_kernel<FMT, T, false, true>);
  return launch_walk(kern, s.grid, st, static_cast<const uint8_t*>(codes),
                     static_cast<const uint8_t*>(scales), rows, cols, s.wx_log2, ts,
                     static_cast<T*>(y), ldy);
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
