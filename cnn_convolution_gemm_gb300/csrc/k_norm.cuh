// Norms around a residual block: u = norm_post(z), x' = x + rs g(gate) u, h = norm_pre(x').
//
// Bound by HBM: x and z are read once and x' and h written once; a row stays in
// registers between its up to four reductions (a mean and a sum of squared deviations
// per layer norm: two passes over registers, so that a large mean does not cancel the
// variance's digits).  Blocks that take many rows fetch x and z two rows ahead into shared
// memory (bulk copies); otherwise a row's loads are issued together, past L1, so that the
// weights stay there.  Measured: 32768 x 8192 bf16 325 us (6.6 TB/s), 12544 x 1001 fp32
// with gates 40 us (5.0 TB/s; single elements), 26400 x 256 bf16 with gates 10, 8192 x 4096 bf16
// with fp32 z 66 (5.1 TB/s), one row of 4096 3.1 us.
// One translation unit per set of types includes this file.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "fp4.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace gb {
namespace norm {
using namespace gb::fp4;

// How a row lies over its T threads, N columns each.  SINGLE: single columns at i T + t
// (coalesced at any alignment; the first half of them exists in every thread, since a
// row has more than T N / 2 columns).  Else groups of 16 consecutive columns, group i of
// thread t at 16 (i T + t): GROUPS of rows that allow 32-byte accesses, ANY of others
// (which costs instructions: 12544 x 1001 fp32 79 us, SINGLE 40; for codes, which need
// their blocks in one place).
enum Layout { SINGLE, GROUPS, ANY };
template <int T, int N, Layout L>
struct Lay {
  static constexpr bool VEC = L != SINGLE;
  static constexpr int G = VEC ? N / 16 : N;  // groups
  static constexpr int GC = VEC ? 16 : 1;     // columns of a group
  static __device__ __forceinline__ int col(int i, int t) { return GC * (i * T + t); }
  static __device__ __forceinline__ bool has(int i, int t, int C) {
    return (!VEC && T > 32 && i < N / 2) || col(i, t) < C;
  }
};

// A thread's elements as loaded, from row r of rows.
template <typename E, int T, int N, Layout LAY>
struct RowRegs {
  using L = Lay<T, N, LAY>;
  std::conditional_t<LAY == GROUPS, Raw16<E>, std::conditional_t<LAY == ANY, RawAny16<E>, E>>
      raw[L::G];

  __device__ __forceinline__ void load(const void* t0, long long ld, long long r, long long rows,
                                       int t, int C) {
    const E* const row = static_cast<const E*>(t0) + r * ld;
#pragma unroll
    for (int i = 0; i < L::G; ++i) {
      if constexpr (LAY == GROUPS)
        raw[i].load(row, L::col(i, t), C, true);
      else if constexpr (LAY == ANY)
        raw[i].load(row, L::col(i, t), C, r == 0, r == rows - 1);
      else
        raw[i] = L::has(i, t, C) ? row[L::col(i, t)] : E(0.0f);
    }
  }
  __device__ __forceinline__ void get(float (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < L::G; ++i) {
      if constexpr (LAY != SINGLE) {
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

// The same from a row in shared memory (GROUPS; columns past C read as 0).
template <typename E, int T, int N>
__device__ __forceinline__ void read_shared(float (&v)[N], const uint8_t* row, int t, int C) {
#pragma unroll
  for (int i = 0; i < N / 16; ++i) {
    const int c = 16 * (i * T + t);
    Raw16<E> raw;
#pragma unroll
    for (int k = 0; k < (int)sizeof(E); ++k) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (c + k * (16 / (int)sizeof(E)) < C)  // C is a multiple of 16 bytes of elements
        u = *reinterpret_cast<const uint4*>(row + (size_t)c * sizeof(E) + 16 * k);
      uint32_t* const w = &raw.b[k / 2].w[k % 2 * 4];
      w[0] = u.x;
      w[1] = u.y;
      w[2] = u.z;
      w[3] = u.w;
    }
    float e[16];
    raw.get(e);
#pragma unroll
    for (int k = 0; k < 16; ++k) v[16 * i + k] = e[k];
  }
}

// valid: whether the row exists (lanes of a warp may share it with other rows).
template <typename E, int T, int N, Layout LAY>
__device__ __forceinline__ void store_row(E* row, bool valid, int t, int C, const float (&v)[N]) {
  using L = Lay<T, N, LAY>;
#pragma unroll
  for (int i = 0; i < L::G; ++i) {
    if constexpr (LAY == SINGLE) {
      if (valid && L::has(i, t, C)) store_f32(row + L::col(i, t), v[i]);
    } else {
      float e[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) e[k] = v[16 * i + k];
      const int c0 = L::col(i, t & ~31);  // the warp's first column
      if constexpr (LAY == GROUPS) {
        if (valid) store16(row, L::col(i, t), C, e);
      } else if (c0 < C) {
        store_warp_any16(row, c0, valid ? C : 0, e, t & 31, T < 32 ? T : 32);
      }
    }
  }
}

// Sums over the T threads of each of R rows (a warp, or the block), the same in each
// thread.  red: two buffers used in turn, so that one barrier a sum is enough.
template <int T, int R>
__device__ __forceinline__ void row_sum(float (&v)[R], float (*red)[32 * R], int& turn) {
#pragma unroll
  for (int o = (T < 32 ? T : 32) / 2; o; o >>= 1)
#pragma unroll
    for (int k = 0; k < R; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
  if constexpr (T > 32) {
    constexpr int W = T / 32, P = W <= 2 ? 2 : W <= 4 ? 4 : W <= 8 ? 8 : W <= 16 ? 16 : 32;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < R; ++k)
      if (lane == k) red[turn][32 * k + (threadIdx.x >> 5)] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < R; ++k)
      v[k] = W == P || (lane & (P - 1)) < W ? red[turn][32 * k + (lane & (P - 1))] : 0.0f;
    turn ^= 1;
#pragma unroll
    for (int o = P / 2; o; o >>= 1)
#pragma unroll
      for (int k = 0; k < R; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
  }
}

// Four of the thread's elements of a row of weights or biases (fp32; 0 past the row's
// end), from element k of its N.
template <int T, int N, Layout LAY>
__device__ __forceinline__ float4 load_weights(const float* w, int k, int t, int C, bool vec) {
  using L = Lay<T, N, LAY>;
  float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if constexpr (LAY != SINGLE) {
    const int c = L::col(k / 16, t) + k % 16;
    if (vec && c + 4 <= C) return *reinterpret_cast<const float4*>(w + c);
    if (c < C) f.x = w[c];
    if (c + 1 < C) f.y = w[c + 1];
    if (c + 2 < C) f.z = w[c + 2];
    if (c + 3 < C) f.w = w[c + 3];
  } else {
    if (L::has(k, t, C)) f.x = w[L::col(k, t)];
    if (L::has(k + 1, t, C)) f.y = w[L::col(k + 1, t)];
    if (L::has(k + 2, t, C)) f.z = w[L::col(k + 2, t)];
    if (L::has(k + 3, t, C)) f.w = w[L::col(k + 3, t)];
  }
  return f;
}

// A row of weights or biases.  Blocks that walk over many rows hold each thread's own
// elements in shared memory, four at a time and thread by thread (a thread reads back only
// what it wrote): beside the ring, L1 is too small for them (32768 x 8192 bf16: 35 % of
// the weights' sectors missed, 386 us; a deeper ring was slower still).
template <int T, int N, Layout LAY>
struct Weights {
  const float* w;      // nullptr: none
  const float4* held;  // nullptr: not held

  __device__ __forceinline__ float4 get(int k, int t, int C, bool vec) const {
    return held ? held[k / 4 * T + t] : load_weights<T, N, LAY>(w, k, t, C, vec);
  }
};

// v = norm(v) with weight and bias, for R rows; elements past a row's end come and stay 0.
template <int T, int N, Layout LAY, int R>
__device__ __forceinline__ void norm_rows(float (&v)[R][N], int kind, float eps,
                                          const Weights<T, N, LAY>& w,
                                          const Weights<T, N, LAY>& b, int t, int C, bool vec_w,
                                          float inv, float (*red)[32 * R], int& turn) {
  using L = Lay<T, N, LAY>;
  float sum[R];
  if (kind == CONV_NORM_LAYER) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        s0 += v[k][i];
        s1 += v[k][i + 1];
      }
      sum[k] = s0 + s1;
    }
    row_sum<T, R>(sum, red, turn);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const float mean = sum[k] * inv;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const bool in = LAY != SINGLE ? L::col(i / 16, t) + i % 16 < C : L::has(i, t, C);
        v[k][i] = in ? v[k][i] - mean : 0.0f;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < R; ++k) {
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      s0 = fmaf(v[k][i], v[k][i], s0);
      s1 = fmaf(v[k][i + 1], v[k][i + 1], s1);
    }
    sum[k] = s0 + s1;
  }
  row_sum<T, R>(sum, red, turn);
  float f[R];
#pragma unroll
  for (int k = 0; k < R; ++k) f[k] = rsqrtf(fmaf(sum[k], inv, eps));
  if (w.w) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 e = w.get(i, t, C, vec_w);
#pragma unroll
      for (int k = 0; k < R; ++k) {
        v[k][i] *= f[k] * e.x;
        v[k][i + 1] *= f[k] * e.y;
        v[k][i + 2] *= f[k] * e.z;
        v[k][i + 3] *= f[k] * e.w;
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int i = 0; i < N; ++i) v[k][i] *= f[k];
  }
  if (b.w) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 e = b.get(i, t, C, vec_w);
#pragma unroll
      for (int k = 0; k < R; ++k) {
        v[k][i] += e.x;
        v[k][i + 1] += e.y;
        v[k][i + 2] += e.z;
        v[k][i + 3] += e.w;
      }
    }
  }
}

constexpr int RING = 2;  // stages of R rows in shared memory

// Stores h of one row.
template <typename TG, int T, int N, Layout LAY>
__device__ __forceinline__ void store_h(const NormArgs& a, const TensorScale& ts, long long r,
                                        int t, const float (&v)[N]) {
  const bool valid = T >= 32 || r < a.rows;
  const int C = a.C;
  if (a.out == CONV_NORM_OUT_FLOAT) {
    store_row<TG, T, N, LAY>(static_cast<TG*>(a.h) + r * a.ldh, valid, t, C, v);
  } else if constexpr (LAY != SINGLE) {
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
      uint2 packed;
      uint32_t word;
      uint8_t* const codes = static_cast<uint8_t*>(a.h);
      const int c = 16 * (i * T + t);
      if (a.out == CONV_NORM_OUT_FP4_MX) {
        quantize16<CONV_FP4_MX>(e, ts, packed, word);
        if (valid) store_quantized16<CONV_FP4_MX>(packed, word, r, c, C, codes, a.hs);
      } else {
        quantize16<CONV_FP4_NV>(e, ts, packed, word);
        if (valid) store_quantized16<CONV_FP4_NV>(packed, word, r, c, C, codes, a.hs);
      }
    }
  }
}

// Blocks an SM has to hold, which caps the registers: the compiler otherwise spends more on
// loads it spreads between the sums (8192 x 4096 with gates 52 us, uncapped 74; 14552 x 2579
// bf16 145, 223).  Without z more fit: 16384 x 8192 bf16 to MX 106 -> 91 us.
constexpr int least_blocks(int T, int N, Layout lay, bool ahead, int R, bool has_z) {
  const int block = T <= 32 ? 128 : T;
  int threads = 1;
  if (ahead)
    threads = T % 192 == 0 || (T == 256 && R == 1) ? 768 : has_z ? 512 : 1024;
  else if (N == 8)
    threads = has_z ? (T >= 512 ? 1024 : 768) : 1;
  else if (N == 16)
    threads = lay == ANY ? 1 : 512;
  return threads > block ? threads / block : 1;
}

// T <= 32: 32 / T rows per warp (4 warps in a block), else R rows at a time per block of T
// threads.
// AHEAD (GROUPS, T > 32): x and z (if given) come through the ring; else R is 1.
// HASZ false: z is not given (the first norm of a network or block).
// Types: TX of x and x', TZ of z, TG of the gates and h.
// vec_w: 16-byte accesses to weights.  held: how many of their rows shared memory has room for.
template <typename TX, typename TZ, typename TG, int T, int N, Layout LAY, bool AHEAD, int R,
          bool HASZ>
__global__ void __launch_bounds__(T <= 32 ? 128 : T, least_blocks(T, N, LAY, AHEAD, R, HASZ))
    norm_kernel(const NormArgs a, const TensorScale ts, const bool vec_w, const int held) {
  static_assert(AHEAD ? LAY == GROUPS : R == 1, "rows of a step");
  __shared__ float red[2][32 * R];
  __shared__ uint64_t full[RING];
  extern __shared__ uint4 ring[];  // RING x R x (a row of z, a row of x); weights
  gb::allow_dependents();
  const int C = a.C;
  constexpr bool FP32 = sizeof(TX) == 4 || sizeof(TG) == 4;  // outputs of 32 bits
  constexpr int AT_ONCE = T <= 32 ? 128 / T : R;  // rows of a block
  const int t = T <= 32 ? (int)threadIdx.x & (T - 1) : (int)threadIdx.x;
  const long long step = (long long)gridDim.x * AT_ONCE;
  const long long first =
      (long long)blockIdx.x * AT_ONCE + (T <= 32 ? (int)threadIdx.x / T : 0);
  // the lanes of a warp go round together, as long as its first row exists
  const int after = T < 32 ? (int)(threadIdx.x & 31) / T : 0;
  const float inv = 1.0f / (float)C;
  const uint32_t zb = HASZ ? (uint32_t)C * sizeof(TZ) : 0u, xb = (uint32_t)C * sizeof(TX);
  const auto fetch = [&](long long r, int stage) {  // one thread
    uint8_t* to = reinterpret_cast<uint8_t*>(ring) + stage * (size_t)(zb + xb) * R;
    const int rows = (int)(a.rows - r < R ? a.rows - r : R);
    gb::mbar_arrive_expect_tx(&full[stage], (zb + xb) * rows);
    for (int k = 0; k < rows; ++k, to += zb + xb) {
      if (HASZ) gb::bulk_load(to, static_cast<const TZ*>(a.z) + (r + k) * a.ldz, &full[stage], zb);
      gb::bulk_load(to + zb, static_cast<const TX*>(a.x) + (r + k) * a.ldx, &full[stage], xb);
    }
  };
  Weights<T, N, LAY> w_post{a.w_post, nullptr}, b_post{a.b_post, nullptr},
      w_pre{a.w_pre, nullptr}, b_pre{a.b_pre, nullptr};
  if (AHEAD && t == 0) {
    for (int i = 0; i < RING; ++i) gb::mbar_init(&full[i], 1);
    gb::fence_barrier_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (AHEAD) {
    if (t == 0)
      for (int i = 0; i < RING && first + i * step < a.rows; ++i) fetch(first + i * step, i);
    float4* to = reinterpret_cast<float4*>(reinterpret_cast<uint8_t*>(ring) +
                                           RING * R * (size_t)(zb + xb));
    int room = held;
    const auto hold = [&](Weights<T, N, LAY>& w) {
      if (!w.w || room-- <= 0) return;
#pragma unroll
      for (int k = 0; k < N; k += 4)
        to[k / 4 * T + t] = load_weights<T, N, LAY>(w.w, k, t, C, vec_w);
      w.held = to;
      to += T * N / 4;
    };
    hold(w_post);
    hold(b_post);
    hold(w_pre);
    hold(b_pre);
    __syncthreads();
  }
  const unsigned gates = (unsigned)(a.rows - 1) / (unsigned)a.gate_rows + 1;  // rows of them
  int turn = 0, stage = 0;
  uint32_t phase = 0;
  bool ok = true;  // after a wait that ran out nothing is waited for again (the rows are
                   // then wrong, and the error word says so); the barriers stay in step, and
                   // stage and phase those of the copies that are still on their way
  // without the ring: the next row's z and x are on their way from the moment on that
  // their registers are free (12544 x 1001 fp32 40 -> 38 us, 14552 x 2579 146 -> 134; rows
  // above 8192 have none to spare: 2656 x 12544 fp32 176, so 214)
  constexpr bool NEXT = !AHEAD && N <= 16 && T * N <= 8192;
  RowRegs<TX, T, N, LAY> next_x;
  RowRegs<TZ, T, N, LAY> next_z;
  const auto load_z = [&](RowRegs<TZ, T, N, LAY>& to, long long r) {
    if (HASZ && r < a.rows) to.load(a.z, a.ldz, r, a.rows, t, C);
  };
  const auto load_x = [&](RowRegs<TX, T, N, LAY>& to, long long r) {
    if (r < a.rows) to.load(a.x, a.ldx, r, a.rows, t, C);
  };
  if constexpr (NEXT) {
    load_z(next_z, first);
    load_x(next_x, first);
  }
  for (long long r = first; r - after < a.rows; r += step) {
    const uint8_t* const sz =
        reinterpret_cast<const uint8_t*>(ring) + stage * (size_t)(zb + xb) * R;
    RowRegs<TX, T, N, LAY> own_x;
    RowRegs<TZ, T, N, LAY> own_z;
    RowRegs<TX, T, N, LAY>& rx = NEXT ? next_x : own_x;
    RowRegs<TZ, T, N, LAY>& rz = NEXT ? next_z : own_z;
    if constexpr (!AHEAD && !NEXT) {
      if constexpr (HASZ) rz.load(a.z, a.ldz, r, a.rows, t, C);
      rx.load(a.x, a.ldx, r, a.rows, t, C);
    }
    if (AHEAD && ok) ok = gb::mbar_wait_bounded(&full[stage], phase, a.wait_ns, a.err);
    float v[R][N];
    if constexpr (HASZ) {
      float u[R][N];
      RowRegs<TG, T, N, LAY> rg[R];
#pragma unroll
      for (int k = 0; k < R; ++k) {
        if constexpr (AHEAD)
          read_shared<TZ, T, N>(u[k], sz + k * (zb + xb), t, C);
        else
          rz.get(u[k]);
        if constexpr (NEXT) load_z(rz, r + step);
        if (a.gate_kind != CONV_GATE_NONE) {
          // rows and gate_rows are ints: a 32-bit division
          const unsigned row = (unsigned)(r + k < a.rows ? r + k : a.rows - 1);
          rg[k].load(a.gate, a.ldg, row / (unsigned)a.gate_rows, gates, t, C);
        }
      }
      if (a.post != CONV_NORM_NONE)
        norm_rows<T, N, LAY, R>(u, a.post, a.eps_post, w_post, b_post, t, C, vec_w, inv, red, turn);
#pragma unroll
      for (int k = 0; k < R; ++k) {
        if (a.gate_kind != CONV_GATE_NONE) {
          rg[k].get(v[k]);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            if (a.gate_kind == CONV_GATE_SIGMOID) v[k][i] = logistic<FP32>(v[k][i]);
            u[k][i] *= v[k][i];
          }
        }
        if constexpr (AHEAD)
          read_shared<TX, T, N>(v[k], sz + k * (zb + xb) + zb, t, C);
        else
          rx.get(v[k]);
        if constexpr (NEXT) load_x(rx, r + step);
#pragma unroll
        for (int i = 0; i < N; ++i) v[k][i] = fmaf(a.rs, u[k][i], v[k][i]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < R; ++k) {
        if constexpr (AHEAD)
          read_shared<TX, T, N>(v[k], sz + k * (zb + xb), t, C);
        else
          rx.get(v[k]);
        if constexpr (NEXT) load_x(rx, r + step);
      }
    }
    if (a.x_out) {
#pragma unroll
      for (int k = 0; k < R; ++k)
        if (T < 32 || r + k < a.rows)
          store_row<TX, T, N, LAY>(static_cast<TX*>(a.x_out) + (r + k) * a.ldxo,
                                   T >= 32 || r < a.rows, t, C, v[k]);
    }
    if (a.pre != CONV_NORM_NONE) {
      norm_rows<T, N, LAY, R>(v, a.pre, a.eps_pre, w_pre, b_pre, t, C, vec_w, inv, red, turn);
#pragma unroll
      for (int k = 0; k < R; ++k)
        if (T < 32 || r + k < a.rows) store_h<TG, T, N, LAY>(a, ts, r + k, t, v[k]);
    }
    if constexpr (AHEAD) {
      // every thread has read the rows before a barrier: norm_pre's, or this one
      if (a.pre == CONV_NORM_NONE) __syncthreads();
      if (t == 0 && ok && r + RING * step < a.rows) fetch(r + RING * step, stage);
      if (ok && ++stage == RING) {
        stage = 0;
        phase ^= 1;
      }
    }
  }
  if (AHEAD && t == 0 && !ok) {
    // copies that were on their way when a wait ran out
    for (int i = 0; i < RING; ++i) {
      gb::mbar_wait_bounded(&full[stage], phase, a.wait_ns, a.err);
      if (++stage == RING) {
        stage = 0;
        phase ^= 1;
      }
    }
  }
}

// Blocks of T threads that walk over the rows, as many as the SMs hold.
template <typename K>
cudaError_t launch_rows(K* kern, const NormArgs& a, int block, int rows_per_block, int smem,
                        int held, cudaStream_t st) {
  const long long per_sm = gb_blocks_per_sm(reinterpret_cast<const void*>(kern), block, smem);
  const long long most = (long long)gb_num_sms() * std::max(1LL, per_sm);
  const auto vec = [](const float* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<long long>(gb_ceil_div_ll(a.rows, rows_per_block), most));
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool vec_w = vec(a.w_post) && vec(a.b_post) && vec(a.w_pre) && vec(a.b_pre);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a, tensor_scale(a.h_scale), vec_w, held);
  if (e == cudaSuccess) gb_count_launch();
  return e;
}

template <typename TX, typename TZ, typename TG, int T, int N, Layout LAY>
cudaError_t launch_direct(const NormArgs& a, cudaStream_t st) {
  auto* kern = norm_kernel<TX, TZ, TG, T, N, LAY, false, 1, true>;
  if constexpr (std::is_same_v<TZ, TG>)  // launch(): without z the types are equal
    if (!a.z) kern = norm_kernel<TX, TZ, TG, T, N, LAY, false, 1, false>;
  return launch_rows(kern, a, T <= 32 ? 128 : T, T <= 32 ? 128 / T : 1, 0, 0, st);
}

// 16 consecutive columns a thread up to 8192 channels (152 rows of 4160 bf16 with gates
// 5.4 us, 32 columns 6.7), 32 above
template <typename TX, typename TZ, typename TG, Layout LAY>
cudaError_t launch_groups(const NormArgs& a, cudaStream_t st) {
  if (a.C <= 128) return launch_direct<TX, TZ, TG, 8, 16, LAY>(a, st);
  if (a.C <= 256) return launch_direct<TX, TZ, TG, 16, 16, LAY>(a, st);
  if (a.C <= 512) return launch_direct<TX, TZ, TG, 32, 16, LAY>(a, st);
  if (a.C <= 1024) return launch_direct<TX, TZ, TG, 64, 16, LAY>(a, st);
  if (a.C <= 2048) return launch_direct<TX, TZ, TG, 128, 16, LAY>(a, st);
  if (a.C <= 4096) return launch_direct<TX, TZ, TG, 256, 16, LAY>(a, st);
  if (a.C <= 8192) return launch_direct<TX, TZ, TG, 512, 16, LAY>(a, st);
  if (a.C <= 16384) return launch_direct<TX, TZ, TG, 512, 32, LAY>(a, st);
  return launch_direct<TX, TZ, TG, 1024, 32, LAY>(a, st);
}

// 8 single columns a thread (an access is one element: with more of them registers, not
// bytes on their way, fill the SM: 12544 x 1001 fp32, 16 columns 52 us), 16 and 32 where a
// row needs them
template <typename TX, typename TZ, typename TG>
cudaError_t launch_single(const NormArgs& a, cudaStream_t st) {
  if (a.C <= 256) return launch_direct<TX, TZ, TG, 32, 8, SINGLE>(a, st);
  if (a.C <= 512) return launch_direct<TX, TZ, TG, 64, 8, SINGLE>(a, st);
  if (a.C <= 1024) return launch_direct<TX, TZ, TG, 128, 8, SINGLE>(a, st);
  if (a.C <= 2048) return launch_direct<TX, TZ, TG, 256, 8, SINGLE>(a, st);
  if (a.C <= 4096) return launch_direct<TX, TZ, TG, 512, 8, SINGLE>(a, st);
  if (a.C <= 8192) return launch_direct<TX, TZ, TG, 1024, 8, SINGLE>(a, st);
  if (a.C <= 16384) return launch_direct<TX, TZ, TG, 1024, 16, SINGLE>(a, st);
  return launch_direct<TX, TZ, TG, 1024, 32, SINGLE>(a, st);
}

// Shared memory of the ring and the weights beside it; the latter as far as they fit.
struct AheadSmem {
  int bytes, held;
  bool all, twice;  // all weights; and two blocks on an SM
};
template <typename TX, typename TZ, int T, int R>
AheadSmem ahead_smem(const NormArgs& a) {
  const int most = 224 * 1024, row = T * 64;
  const int n = (a.w_post != nullptr) + (a.b_post != nullptr) + (a.w_pre != nullptr) +
                (a.b_pre != nullptr);
  const int ring = RING * R * a.C * (int)(sizeof(TX) + (a.z ? sizeof(TZ) : 0));
  if (ring > most) return {};
  const int held = std::min(n, (most - ring) / row);
  const int bytes = ring + held * row;
  return {bytes, held, held == n, held == n && 2 * bytes <= most};
}

// Z_ONLY: called with z alone.
template <typename TX, typename TZ, typename TG, int T, int R, bool Z_ONLY = false>
cudaError_t launch_ahead(const NormArgs& a, cudaStream_t st) {
  auto* kern = norm_kernel<TX, TZ, TG, T, 16, GROUPS, true, R, true>;
  if constexpr (!Z_ONLY && std::is_same_v<TZ, TG>)
    if (!a.z) kern = norm_kernel<TX, TZ, TG, T, 16, GROUPS, true, R, false>;
  const AheadSmem smem = ahead_smem<TX, TZ, T, R>(a);
  const cudaError_t e = gb_set_smem_once(reinterpret_cast<const void*>(kern), smem.bytes);
  if (e != cudaSuccess) return e;
  return launch_rows(kern, a, T, R, smem.bytes, smem.held, st);
}

template <typename TX, typename TZ, typename TG = TZ>
cudaError_t launch(const NormArgs& a, cudaStream_t st) {
  if constexpr (!std::is_same_v<TZ, TG>)
    if (!a.z) return cudaErrorInvalidValue;  // the caller's to dispatch by TX and TG
  const bool codes = a.out != CONV_NORM_OUT_FLOAT;
  const auto fit_x = [](const void* p, long long ld) { return !p || rows_vec<TX>(p, ld, 32); };
  const auto fit_z = [](const void* p, long long ld) { return !p || rows_vec<TZ>(p, ld, 32); };
  const auto fit_g = [](const void* p, long long ld) { return !p || rows_vec<TG>(p, ld, 32); };
  const bool vec = fit_x(a.x, a.ldx) && fit_x(a.x_out, a.ldxo) && fit_z(a.z, a.ldz) &&
                   fit_g(a.gate, a.ldg) && (codes || fit_g(a.h, a.ldh));
  // many rows of whole 16-byte pieces: through the ring, two at a time where they fit.  Above
  // 4096 channels three to an SM are many (608 x 8192 bf16 9.3 us, else 10.5; 304 6.3 and
  // 6.1), above 2048 eight, below so many that a block has several steps
  const long long many =
      gb_num_sms() * (a.C > 4096 ? 3LL : a.C > 2048 ? 8LL : 8192 / std::max(a.C, 512) * 8);
  if (vec && a.C > 512 && a.C * sizeof(TX) % 16 == 0 && a.C * sizeof(TZ) % 16 == 0 &&
      a.rows >= many) {
    if (a.C <= 1024) return launch_ahead<TX, TZ, TG, 64, 2>(a, st);
    if (a.C <= 2048) return launch_ahead<TX, TZ, TG, 128, 2>(a, st);
    // one row of 192 threads, four blocks to an SM (12442 x 2560 bf16 46 us, 256 threads and
    // two rows 64)
    if (a.C <= 16 * 192) return launch_ahead<TX, TZ, TG, 192, 1>(a, st);
    if (a.C <= 4096) {
      // likewise (24384 x 4096 bf16, layer norms 220 us, two rows 266; fp32, one block: 427
      // and 343)
      if (a.z && ahead_smem<TX, TZ, 256, 1>(a).twice)
        return launch_ahead<TX, TZ, TG, 256, 1, true>(a, st);
      if (ahead_smem<TX, TZ, 256, 2>(a).all) return launch_ahead<TX, TZ, TG, 256, 2>(a, st);
    } else if (a.C <= 16 * 384 && ahead_smem<TX, TZ, 384, 1>(a).twice) {
      // the same of 384 threads where two blocks fit (12442 x 4768 bf16 93 us, else 125; one
      // block with four weights 200, else 187)
      return launch_ahead<TX, TZ, TG, 384, 1>(a, st);
    } else if (a.C <= 8192) {
      if (ahead_smem<TX, TZ, 512, 2>(a).all) return launch_ahead<TX, TZ, TG, 512, 2>(a, st);
      if (ahead_smem<TX, TZ, 512, 1>(a).all) return launch_ahead<TX, TZ, TG, 512, 1>(a, st);
    } else if (a.C <= 16384 && ahead_smem<TX, TZ, 1024, 1>(a).bytes) {
      return launch_ahead<TX, TZ, TG, 1024, 1>(a, st);
    }
  }
  if (vec) return launch_groups<TX, TZ, TG, GROUPS>(a, st);
  return codes ? launch_groups<TX, TZ, TG, ANY>(a, st) : launch_single<TX, TZ, TG>(a, st);
}

}  // namespace norm
}  // namespace gb
