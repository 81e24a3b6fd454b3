// Norms around a residual block: u = norm_post(z), x' = x + rs g(gate) u, h = norm_pre(x').
#include <cuda_runtime.h>

#include "fp4.cuh"
#include "internal.h"

namespace {
using namespace gb::fp4;

constexpr int THREADS = 256;

// Sum over the block, the same in every thread.
__device__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < THREADS / 32; ++i) s += red[i];
  return s;
}

// Mean and reciprocal deviation of a row in shared memory: two passes, so that a
// large mean does not cancel the variance's digits.
__device__ void row_stats(const float* row, int C, int kind, float eps, float* red, float& mean,
                          float& rstd) {
  mean = 0.0f;
  float s = 0.0f;
  if (kind == CONV_NORM_LAYER) {
    for (int c = threadIdx.x; c < C; c += THREADS) s += row[c];
    mean = block_sum(s, red) / (float)C;
  }
  s = 0.0f;
  for (int c = threadIdx.x; c < C; c += THREADS) {
    const float d = row[c] - mean;
    s += d * d;
  }
  rstd = 1.0f / sqrtf(block_sum(s, red) / (float)C + eps);
}

// One block per row; the row stays in shared memory as fp32.
template <typename TX, typename TZ>
__global__ void __launch_bounds__(THREADS) norm_kernel(const NormArgs a, const TensorScale ts) {
  extern __shared__ float row[];
  __shared__ float red[THREADS / 32];
  const int C = a.C;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const TX* x = static_cast<const TX*>(a.x) + r * a.ldx;
    if (a.z) {
      const TZ* z = static_cast<const TZ*>(a.z) + r * a.ldz;
      for (int c = threadIdx.x; c < C; c += THREADS) row[c] = load_f32(z + c);
      __syncthreads();
      float mean = 0.0f, rstd = 1.0f;
      if (a.post != CONV_NORM_NONE) row_stats(row, C, a.post, a.eps_post, red, mean, rstd);
      const TZ* gate = a.gate_kind == CONV_GATE_NONE
                           ? nullptr
                           : static_cast<const TZ*>(a.gate) + (r / a.gate_rows) * a.ldg;
      for (int c = threadIdx.x; c < C; c += THREADS) {
        float u = (row[c] - mean) * rstd;
        if (a.post != CONV_NORM_NONE) {
          if (a.w_post) u *= a.w_post[c];
          if (a.b_post) u += a.b_post[c];
        }
        float g = a.rs;
        if (gate) {
          const float v = load_f32(gate + c);
          g *= a.gate_kind == CONV_GATE_SIGMOID ? 1.0f / (1.0f + expf(-v)) : v;
        }
        row[c] = load_f32(x + c) + g * u;
      }
    } else {
      for (int c = threadIdx.x; c < C; c += THREADS) row[c] = load_f32(x + c);
    }
    __syncthreads();
    if (a.x_out) {
      TX* xo = static_cast<TX*>(a.x_out) + r * a.ldxo;
      for (int c = threadIdx.x; c < C; c += THREADS) store_f32(xo + c, row[c]);
    }
    if (a.pre != CONV_NORM_NONE) {
      float mean, rstd;
      row_stats(row, C, a.pre, a.eps_pre, red, mean, rstd);
      const int end = a.out == CONV_NORM_OUT_FLOAT ? C : (C + 255) / 256 * 256;
      for (int c0 = (threadIdx.x >> 5) * 256; c0 < end; c0 += THREADS * 8) {
        const int c = c0 + (threadIdx.x & 31) * 8;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = 0.0f;
          if (c + i >= C) continue;
          v[i] = (row[c + i] - mean) * rstd;
          if (a.w_pre) v[i] *= a.w_pre[c + i];
          if (a.b_pre) v[i] += a.b_pre[c + i];
        }
        if (a.out == CONV_NORM_OUT_FLOAT)
          store8(static_cast<TZ*>(a.h) + r * a.ldh, c, C, false, v);
        else if (a.out == CONV_NORM_OUT_FP4_MX)
          store_warp_row<CONV_FP4_MX>(v, ts, r, c0, C, static_cast<uint8_t*>(a.h), a.hs);
        else
          store_warp_row<CONV_FP4_NV>(v, ts, r, c0, C, static_cast<uint8_t*>(a.h), a.hs);
      }
    }
    __syncthreads();
  }
}

template <typename TX, typename TZ>
cudaError_t norm_t(const NormArgs& a, cudaStream_t st) {
  auto* kern = norm_kernel<TX, TZ>;
  const int smem = a.C * 4;
  const cudaError_t e = gb_set_smem_once(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  const int most = gb_num_sms() * 8;
  kern<<<a.rows < most ? a.rows : most, THREADS, smem, st>>>(a, tensor_scale(a.h_scale));
  gb_count_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, cudaStream_t st) {
  if (a.x_dtype == CONV_BF16)
    return a.z_dtype == CONV_BF16 ? norm_t<__nv_bfloat16, __nv_bfloat16>(a, st)
                                  : norm_t<__nv_bfloat16, float>(a, st);
  return a.z_dtype == CONV_BF16 ? norm_t<float, __nv_bfloat16>(a, st) : norm_t<float, float>(a, st);
}
