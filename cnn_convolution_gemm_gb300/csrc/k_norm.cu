// Norms around a residual block: u = norm_post(z), x' = x + rs g(gate) u, h = norm_pre(x').
//
// Bound by HBM: x and z are read once and x' and h written once; a row stays in
// registers between its up to four reductions (a mean and a sum of squared deviations
// per layer norm: two passes over registers, so that a large mean does not cancel the
// variance's digits).  The loads of a row are issued together; several blocks on an SM
// cover each other's reductions.  x and z pass L1 by, so that the weights stay there.
#include <cuda_runtime.h>

#include <algorithm>

#include "fp4.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace {
using namespace gb::fp4;

// Sum over the threads of a row (a warp, or the block), the same in each.  red: two
// buffers used in turn, so that one barrier a sum is enough.
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float (*red)[32], int& turn) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if constexpr (WARP) return v;
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) red[turn][threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? red[turn][lane] : 0.0f;
  turn ^= 1;
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Loads that do not displace the weights in L1.
__device__ __forceinline__ uint4 load_stream16(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// A thread's elements of a row.  VEC: groups of 8 consecutive columns (16-byte
// accesses where vec says so), group i at 8 (i * threads + t); else single columns
// t, t + threads, .. (coalesced at any alignment).
template <typename T, int N, bool VEC>
__device__ __forceinline__ void load_row(const T* row, int t, int threads, int C, bool vec,
                                         float (&v)[N]) {
  if constexpr (VEC) {
    if (vec) {
      uint4 raw[N / 8][sizeof(T) / 2];
#pragma unroll
      for (int i = 0; i < N / 8; ++i) {
        const int c = 8 * (i * threads + t);
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k)
          raw[i][k] = c < C ? load_stream16(row + c + k * (16 / (int)sizeof(T)))
                            : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < N / 8; ++i) {
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k) {
          const uint32_t w[4] = {raw[i][k].x, raw[i][k].y, raw[i][k].z, raw[i][k].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (sizeof(T) == 2) {
              v[i * 8 + 2 * j] = __uint_as_float(w[j] << 16);
              v[i * 8 + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            } else {
              v[i * 8 + 4 * k + j] = __uint_as_float(w[j]);
            }
          }
        }
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = 8 * (i / 8 * threads + t) + i % 8;
      v[i] = c < C ? load_f32(row + c) : 0.0f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = i * threads + t;
      v[i] = c < C ? load_f32(row + c) : 0.0f;
    }
  }
}

template <typename T, int N, bool VEC>
__device__ __forceinline__ void store_row(T* row, int t, int threads, int C, bool vec,
                                          const float (&v)[N]) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      float e[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) e[k] = v[i * 8 + k];
      store8(row, 8 * (i * threads + t), C, vec, e);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = i * threads + t;
      if (c < C) store_f32(row + c, v[i]);
    }
  }
}

// v = norm(v) with weight and bias; columns past C are left at 0.
template <int N, bool VEC, bool WARP>
__device__ __forceinline__ void norm_row(float (&v)[N], int kind, float eps, const float* w,
                                         const float* b, int t, int threads, int C, bool vec_w,
                                         float (*red)[32], int& turn) {
  const float inv = 1.0f / (float)C;
  if (kind == CONV_NORM_LAYER) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) s += v[i];
    const float mean = row_sum<WARP>(s, red, turn) * inv;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = VEC ? 8 * (i / 8 * threads + t) + i % 8 : i * threads + t;
      v[i] = c < C ? v[i] - mean : 0.0f;
    }
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) s = fmaf(v[i], v[i], s);
  const float rstd = 1.0f / sqrtf(row_sum<WARP>(s, red, turn) * inv + eps);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] *= rstd;
  for (int k = 0; k < 2; ++k) {
    const float* const a = k == 0 ? w : b;
    if (!a) continue;
    if (VEC && vec_w) {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const int c = 8 * (i / 8 * threads + t) + i % 8;
        if (c >= C) continue;
        const float4 f = *reinterpret_cast<const float4*>(a + c);
        const float e[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i + j] = k == 0 ? v[i + j] * e[j] : v[i + j] + e[j];
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = VEC ? 8 * (i / 8 * threads + t) + i % 8 : i * threads + t;
        if (c < C) v[i] = k == 0 ? v[i] * a[c] : v[i] + a[c];
      }
    }
  }
}

// WARP: one row per warp (4 in a block), else one per block of up to MAXT threads.
// N columns a thread.
template <typename TX, typename TZ, int N, bool VEC, bool WARP, int MAXT>
__global__ void __launch_bounds__(MAXT)
    norm_kernel(const NormArgs a, const TensorScale ts, int vec_x, int vec_z, int vec_g, int vec_xo,
                int vec_h, int vec_w) {
  __shared__ float red[2][32];
  gb::allow_dependents();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int C = a.C, threads = WARP ? 32 : (int)blockDim.x;
  const int t = WARP ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
  const long long step = WARP ? gridDim.x * 4LL : gridDim.x;
  int turn = 0;
  for (long long r = WARP ? blockIdx.x * 4LL + (threadIdx.x >> 5) : blockIdx.x; r < a.rows;
       r += step) {
    float x[N], u[N];
    if (a.z)
      load_row<TZ, N, VEC>(static_cast<const TZ*>(a.z) + r * a.ldz, t, threads, C, vec_z, u);
    load_row<TX, N, VEC>(static_cast<const TX*>(a.x) + r * a.ldx, t, threads, C, vec_x, x);
    if (a.z) {
      if (a.post != CONV_NORM_NONE)
        norm_row<N, VEC, WARP>(u, a.post, a.eps_post, a.w_post, a.b_post, t, threads, C, vec_w, red,
                               turn);
      if (a.gate_kind != CONV_GATE_NONE) {
        float g[N];
        load_row<TZ, N, VEC>(static_cast<const TZ*>(a.gate) + r / a.gate_rows * a.ldg, t, threads,
                             C, vec_g, g);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          // the logistic function within 2^-21
          if (a.gate_kind == CONV_GATE_SIGMOID)
            g[i] = rcp_approx(1.0f + ex2_approx(g[i] * -1.4426950408889634f));
          x[i] = fmaf(a.rs * g[i], u[i], x[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = fmaf(a.rs, u[i], x[i]);
      }
    }
    if (a.x_out)
      store_row<TX, N, VEC>(static_cast<TX*>(a.x_out) + r * a.ldxo, t, threads, C, vec_xo, x);
    if (a.pre == CONV_NORM_NONE) continue;
    norm_row<N, VEC, WARP>(x, a.pre, a.eps_pre, a.w_pre, a.b_pre, t, threads, C, vec_w, red, turn);
    if (a.out == CONV_NORM_OUT_FLOAT) {
      store_row<TZ, N, VEC>(static_cast<TZ*>(a.h) + r * a.ldh, t, threads, C, vec_h, x);
    } else if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < N / 8; ++i) {
        const int c0 = 8 * (i * threads + (t & ~31));  // the warp's first column
        if (c0 >= C) break;
        float e[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k] = x[i * 8 + k];
        if (a.out == CONV_NORM_OUT_FP4_MX)
          store_warp_row<CONV_FP4_MX>(e, ts, r, c0, C, static_cast<uint8_t*>(a.h), a.hs);
        else
          store_warp_row<CONV_FP4_NV>(e, ts, r, c0, C, static_cast<uint8_t*>(a.h), a.hs);
      }
    }
  }
}

template <typename TX, typename TZ, int N, bool VEC, bool WARP, int MAXT>
cudaError_t launch_t(const NormArgs& a, int threads, cudaStream_t st) {
  auto* kern = norm_kernel<TX, TZ, N, VEC, WARP, MAXT>;
  // C a multiple of 8, so that no 16-byte access of a row passes its end
  const bool c8 = a.C % 8 == 0;
  const auto vec_w = [&](const float* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  const int block = WARP ? 128 : threads;
  const int rows = WARP ? 4 : 1;
  // as many blocks as the SMs hold: each then walks over rows
  const long long most = (long long)gb_num_sms() * (2048 / block);
  const long long blocks = std::min<long long>(gb_ceil_div_ll(a.rows, rows), most);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3((unsigned)block);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(
      &cfg, kern, a, tensor_scale(a.h_scale), (int)(c8 && rows_vec<TX>(a.x, a.ldx)),
      (int)(c8 && rows_vec<TZ>(a.z, a.ldz)), (int)(c8 && rows_vec<TZ>(a.gate, a.ldg)),
      (int)(c8 && rows_vec<TX>(a.x_out, a.ldxo)), (int)(c8 && rows_vec<TZ>(a.h, a.ldh)),
      (int)(c8 && vec_w(a.w_post) && vec_w(a.b_post) && vec_w(a.w_pre) && vec_w(a.b_pre)));
  if (e == cudaSuccess) gb_count_launch();
  return e;
}

template <typename TX, typename TZ, bool VEC>
cudaError_t launch_c(const NormArgs& a, cudaStream_t st) {
  // 16 columns a thread (8 up to 256 channels, 32 above 16384, where registers spill), a
  // power of two of threads from a warp to 1024
  if (a.C <= 256) return launch_t<TX, TZ, 8, VEC, true, 128>(a, 32, st);
  if (a.C <= 512) return launch_t<TX, TZ, 16, VEC, true, 128>(a, 32, st);
  if (a.C > 16384) return launch_t<TX, TZ, 32, VEC, false, 1024>(a, 1024, st);
  if (a.C > 8192) return launch_t<TX, TZ, 16, VEC, false, 1024>(a, 1024, st);
  int threads = 64;
  while (threads * 16 < a.C) threads *= 2;
  return launch_t<TX, TZ, 16, VEC, false, 512>(a, threads, st);
}

template <typename TX, typename TZ>
cudaError_t launch_types(const NormArgs& a, cudaStream_t st) {
  // 8 consecutive columns a thread where that makes 16-byte accesses, or codes
  const bool vec = a.C % 8 == 0 && rows_vec<TX>(a.x, a.ldx) && (!a.z || rows_vec<TZ>(a.z, a.ldz));
  return vec || a.out != CONV_NORM_OUT_FLOAT ? launch_c<TX, TZ, true>(a, st)
                                             : launch_c<TX, TZ, false>(a, st);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, cudaStream_t st) {
  if (a.x_dtype == CONV_BF16)
    return a.z_dtype == CONV_BF16 ? launch_types<__nv_bfloat16, __nv_bfloat16>(a, st)
                                  : launch_types<__nv_bfloat16, float>(a, st);
  return a.z_dtype == CONV_BF16 ? launch_types<float, __nv_bfloat16>(a, st)
                                : launch_types<float, float>(a, st);
}
