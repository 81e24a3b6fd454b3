// Norms around a residual block: u = norm_post(z), x' = x + rs g(gate) u, h = norm_pre(x').
//
// Bound by HBM: x and z are read once and x' and h written once; a row stays in
// registers between its up to four reductions (a mean and a sum of squared deviations
// per layer norm: two passes over registers, so that a large mean does not cancel the
// variance's digits).  The loads of a row are issued together; several blocks on an SM
// cover each other's reductions.  x and z pass L1 by, so that the weights stay there.
// One translation unit per pair of types includes this file.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>

#include "fp4.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace gb {
namespace norm {
using namespace gb::fp4;

// How a row lies over its T threads, N columns each.  VEC: groups of 16 consecutive
// columns, group i of thread t at 16 (i T + t); else single columns at i T + t
// (coalesced at any alignment; the first half of them exists in every thread, since a
// row has more than T N / 2 columns).
template <int T, int N, bool VEC>
struct Lay {
  static constexpr int G = VEC ? N / 16 : N;  // groups
  static constexpr int GC = VEC ? 16 : 1;     // columns of a group
  static __device__ __forceinline__ int col(int i, int t) { return GC * (i * T + t); }
  static __device__ __forceinline__ bool has(int i, int t, int C) {
    return (!VEC && T > 32 && i < N / 2) || col(i, t) < C;
  }
};

// A thread's elements as loaded.
template <typename E, int T, int N, bool VEC>
struct RowRegs {
  using L = Lay<T, N, VEC>;
  std::conditional_t<VEC, Raw16<E>, E> raw[L::G];

  __device__ __forceinline__ void load(const E* row, int t, int C, bool vec) {
#pragma unroll
    for (int i = 0; i < L::G; ++i) {
      if constexpr (VEC)
        raw[i].load(row, L::col(i, t), C, vec);
      else
        raw[i] = L::has(i, t, C) ? row[L::col(i, t)] : E(0.0f);
    }
  }
  __device__ __forceinline__ void get(float (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < L::G; ++i) {
      if constexpr (VEC) {
        float e[16];
        raw[i].get(e);
#pragma unroll
        for (int k = 0; k < 16; ++k) v[16 * i + k] = e[k];
      } else {
        v[i] = load_f32(&raw[i]);
      }
    }
  }
};

template <typename E, int T, int N, bool VEC>
__device__ __forceinline__ void store_row(E* row, int t, int C, bool vec, const float (&v)[N]) {
  using L = Lay<T, N, VEC>;
#pragma unroll
  for (int i = 0; i < L::G; ++i) {
    if constexpr (VEC) {
      float e[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) e[k] = v[16 * i + k];
      store16(row, L::col(i, t), C, vec, e);
    } else {
      if (L::has(i, t, C)) store_f32(row + L::col(i, t), v[i]);
    }
  }
}

// Sum over the T threads of a row (a warp, or the block), the same in each.  red: two
// buffers used in turn, so that one barrier a sum is enough.
template <int T>
__device__ __forceinline__ float row_sum(float v, float (*red)[32], int& turn) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if constexpr (T > 32) {
    constexpr int W = T / 32;
    const int lane = threadIdx.x & 31;
    if (lane == 0) red[turn][threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[turn][lane & (W - 1)];
    turn ^= 1;
#pragma unroll
    for (int o = W / 2; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  }
  return v;
}

// v = v * f * w (scale and weight) or v + b, w or b a row of fp32 that stays in L1
template <int T, int N, bool VEC, bool ADD>
__device__ __forceinline__ void apply(float (&v)[N], float f, const float* w, int t, int C,
                                      bool vec) {
  using L = Lay<T, N, VEC>;
  const uint64_t f2 = pack2(f, f);
#pragma unroll
  for (int i = 0; i < L::G; ++i) {
    const int c = L::col(i, t);
    if constexpr (VEC) {
#pragma unroll
      for (int k = 0; k < 16; k += 4) {
        float4 e = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (vec && c + 16 <= C) {
          e = *reinterpret_cast<const float4*>(w + c + k);
        } else {
          if (c + k < C) e.x = w[c + k];
          if (c + k + 1 < C) e.y = w[c + k + 1];
          if (c + k + 2 < C) e.z = w[c + k + 2];
          if (c + k + 3 < C) e.w = w[c + k + 3];
        }
        float* const a = &v[16 * i + k];
        if (ADD) {
          a[0] += e.x;
          a[1] += e.y;
          a[2] += e.z;
          a[3] += e.w;
        } else {
          unpack2(mul2(mul2(pack2(a[0], a[1]), f2), pack2(e.x, e.y)), a[0], a[1]);
          unpack2(mul2(mul2(pack2(a[2], a[3]), f2), pack2(e.z, e.w)), a[2], a[3]);
        }
      }
    } else {
      const float e = L::has(i, t, C) ? w[c] : 0.0f;
      v[i] = ADD ? v[i] + e : v[i] * f * e;
    }
  }
}

// v = norm(v) with weight and bias; elements past the row's end come and stay 0.
template <int T, int N, bool VEC>
__device__ __forceinline__ void norm_row(float (&v)[N], int kind, float eps, const float* w,
                                         const float* b, int t, int C, bool vec_w, float inv,
                                         float (*red)[32], int& turn) {
  using L = Lay<T, N, VEC>;
  if (kind == CONV_NORM_LAYER) {
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      s0 += v[i];
      s1 += v[i + 1];
    }
    const float mean = row_sum<T>(s0 + s1, red, turn) * inv;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool in = VEC ? L::col(i / 16, t) + i % 16 < C : L::has(i, t, C);
      v[i] = in ? v[i] - mean : 0.0f;
    }
  }
  uint64_t s = 0;
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const uint64_t p = pack2(v[i], v[i + 1]);
    s = fma2(p, p, s);
  }
  float s0, s1;
  unpack2(s, s0, s1);
  const float rstd = rsqrtf(fmaf(row_sum<T>(s0 + s1, red, turn), inv, eps));
  if (w) {
    apply<T, N, VEC, false>(v, rstd, w, t, C, vec_w);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= rstd;
  }
  if (b) apply<T, N, VEC, true>(v, 0.0f, b, t, C, vec_w);
}

struct Vec {
  bool x, z, g, xo, h, w;  // 32-byte accesses to rows; 16-byte ones to weights
};

// T == 32: one row per warp (4 in a block), else one per block of T threads.
template <typename TX, typename TZ, int T, int N, bool VEC>
__global__ void __launch_bounds__(T < 128 && T == 32 ? 128 : T)
    norm_kernel(const NormArgs a, const TensorScale ts, const Vec vec) {
  __shared__ float red[2][32];
  gb::allow_dependents();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int C = a.C;
  const int t = T == 32 ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
  const long long step = T == 32 ? gridDim.x * 4LL : gridDim.x;
  const float inv = 1.0f / (float)C;
  int turn = 0;
  for (long long r = T == 32 ? blockIdx.x * 4LL + (threadIdx.x >> 5) : blockIdx.x; r < a.rows;
       r += step) {
    RowRegs<TX, T, N, VEC> rx;
    RowRegs<TZ, T, N, VEC> rz;
    if (a.z) rz.load(static_cast<const TZ*>(a.z) + r * a.ldz, t, C, vec.z);
    rx.load(static_cast<const TX*>(a.x) + r * a.ldx, t, C, vec.x);
    float v[N];
    if (a.z) {
      float u[N];
      rz.get(u);
      if (a.gate_kind != CONV_GATE_NONE)  // in z's place
        rz.load(static_cast<const TZ*>(a.gate) + r / a.gate_rows * a.ldg, t, C, vec.g);
      if (a.post != CONV_NORM_NONE)
        norm_row<T, N, VEC>(u, a.post, a.eps_post, a.w_post, a.b_post, t, C, vec.w, inv, red, turn);
      if (a.gate_kind != CONV_GATE_NONE) {
        rz.get(v);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          // the logistic function within 2^-21
          if (a.gate_kind == CONV_GATE_SIGMOID)
            v[i] = rcp_approx(1.0f + ex2_approx(v[i] * -1.4426950408889634f));
          u[i] *= v[i];
        }
      }
      rx.get(v);
      const uint64_t rs = pack2(a.rs, a.rs);
#pragma unroll
      for (int i = 0; i < N; i += 2)
        unpack2(fma2(pack2(u[i], u[i + 1]), rs, pack2(v[i], v[i + 1])), v[i], v[i + 1]);
    } else {
      rx.get(v);
    }
    if (a.x_out)
      store_row<TX, T, N, VEC>(static_cast<TX*>(a.x_out) + r * a.ldxo, t, C, vec.xo, v);
    if (a.pre == CONV_NORM_NONE) continue;
    norm_row<T, N, VEC>(v, a.pre, a.eps_pre, a.w_pre, a.b_pre, t, C, vec.w, inv, red, turn);
    if (a.out == CONV_NORM_OUT_FLOAT) {
      store_row<TZ, T, N, VEC>(static_cast<TZ*>(a.h) + r * a.ldh, t, C, vec.h, v);
    } else if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < N / 16; ++i) {
        const int c0 = 16 * (i * T + (t & ~31));  // the warp's first column
        if (c0 >= C) break;
        float e[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) e[k] = v[16 * i + k];
        if (16 * (i * T + t) + 16 > C) {  // padding is 0 in a row of NaN too
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (16 * (i * T + t) + k >= C) e[k] = 0.0f;
        }
        if (a.out == CONV_NORM_OUT_FP4_MX)
          store_warp_row<CONV_FP4_MX>(e, ts, r, c0, C, static_cast<uint8_t*>(a.h), a.hs);
        else
          store_warp_row<CONV_FP4_NV>(e, ts, r, c0, C, static_cast<uint8_t*>(a.h), a.hs);
      }
    }
  }
}

template <typename TX, typename TZ, int T, int N, bool VEC>
cudaError_t launch_t(const NormArgs& a, cudaStream_t st) {
  const auto vec_w = [](const float* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  Vec vec;
  vec.x = rows_vec<TX>(a.x, a.ldx, 32);
  vec.z = rows_vec<TZ>(a.z, a.ldz, 32);
  vec.g = rows_vec<TZ>(a.gate, a.ldg, 32);
  vec.xo = rows_vec<TX>(a.x_out, a.ldxo, 32);
  vec.h = rows_vec<TZ>(a.h, a.ldh, 32);
  vec.w = vec_w(a.w_post) && vec_w(a.b_post) && vec_w(a.w_pre) && vec_w(a.b_pre);
  const int block = T == 32 ? 128 : T;
  // as many blocks as the SMs hold: each then walks over rows
  const long long most = (long long)gb_num_sms() * (2048 / block);
  const long long blocks = std::min<long long>(gb_ceil_div_ll(a.rows, T == 32 ? 4 : 1), most);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3((unsigned)block);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, norm_kernel<TX, TZ, T, N, VEC>, a,
                                           tensor_scale(a.h_scale), vec);
  if (e == cudaSuccess) gb_count_launch();
  return e;
}

// 16 columns a thread up to 4096 channels (as few dependent steps as the row allows), 32
// above (a thread's part of the reductions is then a smaller share)
template <typename TX, typename TZ, bool VEC>
cudaError_t launch_c(const NormArgs& a, cudaStream_t st) {
  if (a.C <= 512) return launch_t<TX, TZ, 32, 16, VEC>(a, st);
  if (a.C <= 1024) return launch_t<TX, TZ, 64, 16, VEC>(a, st);
  if (a.C <= 2048) return launch_t<TX, TZ, 128, 16, VEC>(a, st);
  if (a.C <= 4096) return launch_t<TX, TZ, 256, 16, VEC>(a, st);
  if (a.C <= 8192) return launch_t<TX, TZ, 256, 32, VEC>(a, st);
  if (a.C <= 16384) return launch_t<TX, TZ, 512, 32, VEC>(a, st);
  return launch_t<TX, TZ, 1024, 32, VEC>(a, st);
}

template <typename TX, typename TZ>
cudaError_t launch(const NormArgs& a, cudaStream_t st) {
  // 16 consecutive columns a thread where that makes 32-byte loads, or codes
  const bool vec = rows_vec<TX>(a.x, a.ldx, 32) && (!a.z || rows_vec<TZ>(a.z, a.ldz, 32));
  return vec || a.out != CONV_NORM_OUT_FLOAT ? launch_c<TX, TZ, true>(a, st)
                                             : launch_c<TX, TZ, false>(a, st);
}

}  // namespace norm
}  // namespace gb
