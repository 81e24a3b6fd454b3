// 8-bit matrices with scales: quantisation and its inverse.
//
// Bound by HBM.  Scales per 128 columns need nothing but the eight lanes that hold them: a
// walk over the rows.  A scale per row needs the whole row first: it stays in registers
// between the maximum and the codes (columns that do not fit there are read twice, the second
// time from L2).  Measured, 16384 x 8192 bf16 (61 us of bytes): to int8 with scales per 128 76 us,
// back 65; fp32 with scales per row 97 to 105.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"
#include "q8.cuh"
#include "walk.cuh"

namespace {
using namespace gb::fp4;
using namespace gb::walk;
namespace q8 = gb::q8;

template <typename T, bool ANY>
using Raw = std::conditional_t<ANY, RawAny16<T>, Raw16<T>>;

// ANY: rows that 32-byte accesses do not fit
template <typename T, bool ANY>
__device__ __forceinline__ void load_raw(Raw<T, ANY>& raw, const T* x, long long ldx, long long r,
                                         int rows, int c, int cols) {
  if constexpr (ANY)
    raw.load(x + r * ldx, c, cols, r == 0, r == rows - 1);
  else
    raw.load(x + r * ldx, c, cols, true);
}

// Registers for four blocks to an SM, as the bytes on their way need; of fp32, twice the bytes,
// for two.
// LANES: that share a scale.
template <int FMT, typename T, int LANES, bool NARROW, bool ANY>
__global__ void __launch_bounds__(THREADS, sizeof(T) == 2 || ANY ? 4 : 2)
    quantize_groups_kernel(const T* __restrict__ x, long long ldx, int rows, int cols,
                           int wx_log2, uint8_t* __restrict__ codes, float* __restrict__ scales) {
  gb::allow_dependents();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Walk w = walk<NARROW>(wx_log2);
  if (!NARROW && w.c - (int)(threadIdx.x & 31) * 16 >= cols) return;  // the whole warp
  // the lanes of a warp go round together: the shuffles below are the warp's
  const long long lead = w.row - (NARROW ? (threadIdx.x & 31) >> (5 + wx_log2) : 0);
  for (long long r0 = w.row, l0 = lead; l0 < rows; r0 += ROWS * w.step, l0 += ROWS * w.step) {
    Raw<T, ANY> raw[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
      if (r0 + i * w.step < rows)
        load_raw<T, ANY>(raw[i], x, ldx, r0 + i * w.step, rows, w.c, cols);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const long long r = r0 + i * w.step;
      if (l0 + i * w.step >= rows) break;
      float v[16];
      raw[i].get(v);
      q8::store_grouped16<FMT, LANES>(v, r < rows, r, w.c, cols, codes, scales);
    }
  }
}

// A row to the PER threads of a block, 16 columns each at a time, the first HELD of these in
// registers; the next row's are on their way while this one's codes are made.
template <int FMT, typename T, int PER, int HELD, bool ANY>
__global__ void __launch_bounds__(PER, (HELD == 2 ? 768 : 1024) / PER)
    quantize_rows_kernel(const T* __restrict__ x, long long ldx, int rows, int cols,
                         uint8_t* __restrict__ codes, float* __restrict__ scales) {
  constexpr int W = PER / 32;
  __shared__ float red[2][W];
  gb::allow_dependents();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const long long pitch = q8::code_pitch(cols);
  int turn = 0;
  Raw<T, ANY> raw[HELD];
  const auto fetch = [&](long long r) {
    if (r >= rows) return;
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      load_raw<T, ANY>(raw[i], x, ldx, r, rows, 16 * (i * PER + t), cols);
  };
  fetch(blockIdx.x);
  for (long long r = blockIdx.x; r < rows; r += gridDim.x) {
    float v[HELD][16], top = 0.0f;
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      raw[i].get(v[i]);
      top = q8::top16(v[i], top);
    }
    fetch(r + gridDim.x);
    for (int c = 16 * (HELD * PER + t); c < cols; c += 16 * PER) {
      Raw<T, ANY> more;
      float e[16];
      load_raw<T, ANY>(more, x, ldx, r, rows, c, cols);
      more.get(e);
      top = q8::top16(e, top);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = max_abs(top, top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (lane == 0) red[turn][warp] = top;
    __syncthreads();
    top = red[turn][lane % W];
#pragma unroll
    for (int o = W / 2; o; o >>= 1)
      top = max_abs(top, top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    turn ^= 1;  // two buffers used in turn: one barrier is enough
    const q8::Scale<FMT> s(top);
    if (t == 0) scales[r] = s.s;
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const int c = 16 * (i * PER + t);
      if (c < cols) *reinterpret_cast<uint4*>(codes + r * pitch + c) = s.codes16(v[i]);
    }
    for (int c = 16 * (HELD * PER + t); c < cols; c += 16 * PER) {
      Raw<T, ANY> more;
      float e[16];
      load_raw<T, ANY>(more, x, ldx, r, rows, c, cols);
      more.get(e);
      *reinterpret_cast<uint4*>(codes + r * pitch + c) = s.codes16(e);
    }
  }
}

template <int FMT, typename T, bool NARROW, bool ANY>
__global__ void __launch_bounds__(THREADS)
    dequantize_kernel(const uint8_t* __restrict__ codes, const float* __restrict__ scales,
                      int group, int rows, int cols, int wx_log2, T* __restrict__ y,
                      long long ldy) {
  gb::allow_dependents();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Walk w = walk<NARROW>(wx_log2);
  const int lane = NARROW ? w.c / 16 : (int)(threadIdx.x & 31);  // of the row's in this warp
  // ANY: the lanes of a warp hand elements to one another, and go round together
  if (w.c - (ANY ? lane * 16 : 0) >= cols) return;
  const long long lead =
      w.row - (NARROW && ANY ? (int)(threadIdx.x & 31) >> (5 + wx_log2) : 0);
  const long long pitch = q8::code_pitch(cols);
  const int per_row = q8::scales_per_row(group, cols), g = group ? w.c / q8::GROUP : 0;
  for (long long r0 = w.row, l0 = lead; l0 < rows; r0 += ROWS * w.step, l0 += ROWS * w.step) {
    uint4 code[ROWS];
    float s[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const long long r = r0 + i * w.step;
      code[i] = make_uint4(0, 0, 0, 0);
      s[i] = 0.0f;
      if (r >= rows || w.c >= cols) continue;
      code[i] = *reinterpret_cast<const uint4*>(codes + r * pitch + w.c);
      s[i] = scales[r * per_row + g];
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const long long r = r0 + i * w.step;
      if ((ANY ? l0 + i * w.step : r) >= rows) continue;
      float v[16];
      q8::unpack4<FMT>(code[i].x, v);
      q8::unpack4<FMT>(code[i].y, v + 4);
      q8::unpack4<FMT>(code[i].z, v + 8);
      q8::unpack4<FMT>(code[i].w, v + 12);
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] *= s[i];
      if constexpr (ANY)
        store_warp_any16(y + r * ldy, w.c - lane * 16, r < rows ? cols : 0, v, lane,
                         NARROW ? 32 >> -wx_log2 : 32);
      else
        store16(y + r * ldy, w.c, cols, v);
    }
  }
}

template <int FMT, typename T, int PER, int HELD>
cudaError_t quantize_rows(int rows, int cols, const T* x, long long ldx, uint8_t* codes,
                          float* scales, cudaStream_t st) {
  auto* kern = rows_vec<T>(x, ldx, 32) ? quantize_rows_kernel<FMT, T, PER, HELD, false>
                                       : quantize_rows_kernel<FMT, T, PER, HELD, true>;
  const long long per_sm = gb_blocks_per_sm(reinterpret_cast<const void*>(kern), PER, 0);
  const long long most = (long long)gb_num_sms() * std::max(1LL, per_sm);
  return launch_walk<PER>(kern, dim3((unsigned)std::min<long long>(rows, most)), st, x, ldx, rows,
                          cols, codes, scales);
}

template <int FMT, typename T, int LANES, bool NARROW>
cudaError_t quantize_groups(int rows, int cols, const T* x, long long ldx, uint8_t* codes,
                            float* scales, cudaStream_t st) {
  const Shape s = walk_shape(rows, cols);
  auto* kern = rows_vec<T>(x, ldx, 32) ? quantize_groups_kernel<FMT, T, LANES, NARROW, false>
                                       : quantize_groups_kernel<FMT, T, LANES, NARROW, true>;
  return launch_walk(kern, s.grid, st, x, ldx, rows, cols, s.wx_log2, codes, scales);
}

template <int FMT, typename T>
cudaError_t quantize_t(int group, int rows, int cols, const void* xv, long long ldx, void* codes_v,
                       void* scales_v, cudaStream_t st) {
  const T* const x = static_cast<const T*>(xv);
  uint8_t* const codes = static_cast<uint8_t*>(codes_v);
  float* const scales = static_cast<float*>(scales_v);
  // (walk_shape: up to 128 columns on eight lanes, up to 256 on 16, else whole warps)
  if (cols <= 128) return quantize_groups<FMT, T, 8, true>(rows, cols, x, ldx, codes, scales, st);
  if (group)
    return cols <= 256 ? quantize_groups<FMT, T, 8, true>(rows, cols, x, ldx, codes, scales, st)
                       : quantize_groups<FMT, T, 8, false>(rows, cols, x, ldx, codes, scales, st);
  if (cols <= 256) return quantize_groups<FMT, T, 16, true>(rows, cols, x, ldx, codes, scales, st);
  if (cols <= 512) return quantize_groups<FMT, T, 32, false>(rows, cols, x, ldx, codes, scales, st);
  if (cols <= 2048) return quantize_rows<FMT, T, 128, 1>(rows, cols, x, ldx, codes, scales, st);
  if (cols <= 4096) return quantize_rows<FMT, T, 256, 1>(rows, cols, x, ldx, codes, scales, st);
  if (cols <= 8192 && sizeof(T) == 2)
    return quantize_rows<FMT, T, 256, 2>(rows, cols, x, ldx, codes, scales, st);
  if (cols <= 8192) return quantize_rows<FMT, T, 512, 1>(rows, cols, x, ldx, codes, scales, st);
  return quantize_rows<FMT, T, 1024, 1>(rows, cols, x, ldx, codes, scales, st);
}

template <int FMT, typename T>
cudaError_t dequantize_t(int group, int rows, int cols, const void* codes, const void* scales,
                         void* y, long long ldy, cudaStream_t st) {
  const Shape s = walk_shape(rows, cols);
  const bool narrow = s.wx_log2 < 0;
  auto* kern = rows_vec<T>(y, ldy, 32) ? (narrow ? dequantize_kernel<FMT, T, true, false>
                                                 : dequantize_kernel<FMT, T, false, false>)
                                       : (narrow ? dequantize_kernel<FMT, T, true, true>
                                                 : dequantize_kernel<FMT, T, false, true>);
  return launch_walk(kern, s.grid, st, static_cast<const uint8_t*>(codes),
                     static_cast<const float*>(scales), group, rows, cols, s.wx_log2,
                     static_cast<T*>(y), ldy);
}

}  // namespace

cudaError_t launch_q8_quantize(int fmt, int group, int dtype, int rows, int cols, const void* x,
                               long long ldx, void* codes, void* scales, cudaStream_t st) {
  if (fmt == CONV_Q8_E4M3)
    return dtype == CONV_BF16
               ? quantize_t<CONV_Q8_E4M3, __nv_bfloat16>(group, rows, cols, x, ldx, codes, scales,
                                                         st)
               : quantize_t<CONV_Q8_E4M3, float>(group, rows, cols, x, ldx, codes, scales, st);
  return dtype == CONV_BF16
             ? quantize_t<CONV_Q8_INT8, __nv_bfloat16>(group, rows, cols, x, ldx, codes, scales, st)
             : quantize_t<CONV_Q8_INT8, float>(group, rows, cols, x, ldx, codes, scales, st);
}

cudaError_t launch_q8_dequantize(int fmt, int group, int dtype, int rows, int cols,
                                 const void* codes, const void* scales, void* y, long long ldy,
                                 cudaStream_t st) {
  if (fmt == CONV_Q8_E4M3)
    return dtype == CONV_BF16
               ? dequantize_t<CONV_Q8_E4M3, __nv_bfloat16>(group, rows, cols, codes, scales, y,
                                                           ldy, st)
               : dequantize_t<CONV_Q8_E4M3, float>(group, rows, cols, codes, scales, y, ldy, st);
  return dtype == CONV_BF16
             ? dequantize_t<CONV_Q8_INT8, __nv_bfloat16>(group, rows, cols, codes, scales, y, ldy,
                                                         st)
             : dequantize_t<CONV_Q8_INT8, float>(group, rows, cols, codes, scales, y, ldy, st);
}
