// Product of two microscaled 4-bit matrices, y = act(alpha X W^T + bias + residual).
#include <cuda_runtime.h>

#include "fp4.cuh"
#include "internal.h"

namespace {
using namespace gb::fp4;

// One warp per row of X and group of 32 output columns, a column to a lane.
template <int FMT>
__global__ void __launch_bounds__(256) fp4_gemm_simple_kernel(const Fp4Gemm g) {
  const int groups = (g.K + 31) / 32;
  const long long t = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= (long long)g.M * groups) return;
  const long long m = t / groups;
  const int lane = threadIdx.x & 31;
  const int n = (int)(t - m * groups) * 32 + lane;
  const bool live = n < g.K;
  const long long pitch = code_pitch(g.C);
  const int tiles = tiles_per_row(FMT, g.C);
  float acc = 0.0f;
  for (int c = 0; live && c < g.C; c += kBlock<FMT>) {
    const int b = c / kBlock<FMT>;
    const float s =
        scale_value<FMT>(g.xs[scale_word_offset(m, b >> 2, tiles) + (b & 3)], 1.0f) *
        scale_value<FMT>(g.ws[scale_word_offset(n, b >> 2, tiles) + (b & 3)], 1.0f);
    float part = 0.0f;
    for (int i = 0; i < kBlock<FMT>; i += 8) {
      const uint32_t a = *reinterpret_cast<const uint32_t*>(g.x + m * pitch + (c + i) / 2);
      const uint32_t w = *reinterpret_cast<const uint32_t*>(g.w + n * pitch + (c + i) / 2);
      for (int k = 0; k < 8; ++k) part += e2m1_twice(a >> (4 * k) & 15u) * e2m1_twice(w >> (4 * k) & 15u);
    }
    acc += 0.25f * part * s;
  }
  float v = 0.0f;
  if (live) {
    v = acc * g.alpha + (g.bias ? g.bias[n] : 0.0f);
    if (g.res)
      v += g.y_io == CONV_FP4_IO_BF16
               ? load_f32(static_cast<const __nv_bfloat16*>(g.res) + m * g.ldr + n)
               : static_cast<const float*>(g.res)[m * g.ldr + n];
    v = activate(v, g.act);
  }
  if (g.y_io == CONV_FP4_IO_BF16) {
    if (live) store_f32(static_cast<__nv_bfloat16*>(g.y) + m * g.ldy + n, v);
  } else if (g.y_io == CONV_FP4_IO_F32) {
    if (live) static_cast<float*>(g.y)[m * g.ldy + n] = v;
  } else {
    // the 32 columns are the warp's first 4 lanes' eights
    float e[8];
    for (int i = 0; i < 8; ++i) e[i] = __shfl_sync(0xFFFFFFFFu, v, (lane & 3) * 8 + i);
    uint32_t top = 0;
    for (int i = 0; i < 8; ++i) top = max(top, abs_bits(e[i]));
    for (int o = 1; o < kBlock<FMT> / 8; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const BlockScale<FMT> s(__uint_as_float(top), g.y_scale);
    const int c = n - lane + (lane & 3) * 8;
    if (lane < 4)
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(g.y) + m * code_pitch(g.K) + c / 2) =
          s.codes(e);
    const int ot = tiles_per_row(FMT, g.K), b = c / kBlock<FMT>;
    if (lane < 4 && (lane * 8) % kBlock<FMT> == 0 && (b >> 2) < ot)
      g.ys[scale_word_offset(m, b >> 2, ot) + (b & 3)] = (uint8_t)s.byte;
    // the rest of the row's last tile is padding
    if (n - lane + 32 >= g.K && lane == 0)
      for (int pb = (n - lane + 32) / kBlock<FMT>; (pb >> 2) < ot; ++pb)
        g.ys[scale_word_offset(m, pb >> 2, ot) + (pb & 3)] = 0;
  }
}

}  // namespace

cudaError_t launch_fp4_gemm(const Fp4Gemm& g, cudaStream_t st) {
  const long long warps = (long long)g.M * ((g.K + 31) / 32);
  const long long grid = gb_ceil_div_ll(warps, 8);
  if (g.fmt == CONV_FP4_MX)
    fp4_gemm_simple_kernel<CONV_FP4_MX><<<(unsigned)grid, 256, 0, st>>>(g);
  else
    fp4_gemm_simple_kernel<CONV_FP4_NV><<<(unsigned)grid, 256, 0, st>>>(g);
  gb_count_launch();
  return cudaGetLastError();
}
