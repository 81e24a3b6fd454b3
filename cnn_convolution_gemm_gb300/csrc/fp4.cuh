// Device code shared by the kernels that make or read microscaled 4-bit matrices
// (E2M1 codes with one scale per block of 32 or 16 elements; the formats and their
// layout in memory are defined in gbconv.h).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gbconv.h"

namespace gb {
namespace fp4 {

template <int FMT>
constexpr int kBlock = FMT == CONV_FP4_MX ? 32 : 16;

// Tiles of 4 blocks along a row, and bytes between rows of codes.
__host__ __device__ constexpr int tiles_per_row(int fmt, int cols) {
  return fmt == CONV_FP4_MX ? (cols + 127) / 128 : (cols + 63) / 64;
}
__host__ __device__ constexpr long long code_pitch(int cols) {
  return 16LL * ((cols + 31LL) / 32);
}
// Byte offset of the 4 scales of tile tj of row r.
__host__ __device__ constexpr long long scale_word_offset(long long r, int tj, int tiles) {
  return ((r >> 7) * tiles + tj) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

// Eight fp32 values to E2M1 (round to nearest, ties to even, saturating), value i
// in bits 4i..4i+3.
__device__ __forceinline__ uint32_t pack8_e2m1(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 t0, t1, t2, t3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t3, %8, %7;\n\t"
      "mov.b32 %0, {t0, t1, t2, t3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// The value of an E2M1 code, times 2.
__device__ __forceinline__ float e2m1_twice(uint32_t code) {
  const uint32_t m = code & 7u;
  // 0 1 2 3 4 6 8 12: below 4 the code itself, from there (2 + m % 2) << (m / 2 - 1)
  const int t = m < 4u ? (int)m : (int)((2u + (m & 1u)) << ((m >> 1) - 1u));
  return (float)((code & 8u) ? -t : t);
}

// The E4M3 byte nearest to v (>= 0; above 448: 448), and the value of such a byte.
__device__ __forceinline__ uint32_t to_e4m3(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
  return r & 0xFFu;
}
__device__ __forceinline__ float from_e4m3(uint32_t b) {
  const uint32_t e = (b >> 3) & 15u, f = b & 7u;
  if ((b & 0x7Fu) == 0x7Fu) return __int_as_float(0x7FFFFFFF);
  const float a = e ? __uint_as_float(((e + 120u) << 23) | (f << 20)) : (float)f * 0.001953125f;
  return (b & 0x80u) ? -a : a;
}

// The scale byte of a block from its largest magnitude, and the quotients of its
// elements.  NV divides by t = s * tensor_scale: with r = 1 / t rounded to nearest,
// q0 = v r and the exact remainder v - q0 t (one fma) correct each other to the
// rounded quotient (Markstein's correction), so that a quotient that lies on a
// tie of E2M1 arrives there exactly; three operations an element where an IEEE
// division takes about ten.
template <int FMT>
struct BlockScale {
  uint32_t byte;
  float t, r;  // MX: r alone, a power of two

  __device__ __forceinline__ BlockScale(float amax, float tensor_scale) {
    const uint32_t e = __float_as_uint(amax) >> 23;  // amax >= 0 (a NaN: its sign dropped)
    const bool bad = (e & 255u) == 255u;
    if (FMT == CONV_FP4_MX) {
      // floor(log2 amax) = e - 127 for normal numbers; e <= 2 and subnormals: 2^-127
      byte = bad ? 255u : (e > 2u ? e - 2u : 0u);
      r = bad ? 0.0f : __uint_as_float((254u - byte) << 23);  // 2^(127 - byte)
      t = r;
    } else {
      byte = bad ? 0x7Fu : to_e4m3(__fdiv_rn(amax, __fmul_rn(6.0f, tensor_scale)));
      t = bad ? 0.0f : __fmul_rn(from_e4m3(byte), tensor_scale);
      r = __frcp_rn(t);
    }
  }
  // codes of eight elements of the block
  __device__ __forceinline__ uint32_t codes(const float (&v)[8]) const {
    float q[8];
    if (t == 0.0f) return 0u;
    if (FMT == CONV_FP4_MX) {
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = v[i] * r;
    } else if (byte == 0x7Eu) {
      // the largest scale: elements may lie far above 6 t, where the product with r
      // could overflow
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(v[i], t);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float q0 = v[i] * r;
        q[i] = __fmaf_rn(__fmaf_rn(-q0, t, v[i]), r, q0);
      }
    }
    return pack8_e2m1(q);
  }
};

// The factor of a stored scale byte: the value of a code is E2M1 * factor.
template <int FMT>
__device__ __forceinline__ float scale_value(uint32_t byte, float tensor_scale) {
  if (FMT == CONV_FP4_MX) {
    if (byte == 255u) return __int_as_float(0x7FFFFFFF);
    return byte ? __uint_as_float(byte << 23) : __uint_as_float(0x00400000u);  // 2^(byte - 127)
  }
  return __fmul_rn(from_e4m3(byte), tensor_scale);
}

// max of magnitudes that keeps a NaN: compared as bit patterns, where every NaN
// and infinity lies above every finite magnitude.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// One warp turns 256 consecutive columns of a row, eight to a lane (v; zero past
// the last column), into codes and scales.  c0: the warp's first column.  All lanes
// call it.  MX: 4 lanes share a block and 16 a scale tile; NV: 2 and 8.
template <int FMT>
__device__ __forceinline__ void store_warp_row(const float (&v)[8], float tensor_scale, long long r,
                                               int c0, int cols, uint8_t* __restrict__ codes,
                                               uint8_t* __restrict__ scales) {
  const int lane = threadIdx.x & 31;
  constexpr int LB = kBlock<FMT> / 8;  // lanes per block
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, abs_bits(v[i]));
#pragma unroll
  for (int o = 1; o < LB; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  const BlockScale<FMT> s(__uint_as_float(top), tensor_scale);
  const uint32_t packed = s.codes(v);
  uint32_t word = s.byte << (8 * ((lane / LB) & 3));
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, LB);
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2 * LB);
  const int c = c0 + lane * 8;
  const long long pitch = code_pitch(cols);
  if (c < 2 * pitch) *reinterpret_cast<uint32_t*>(codes + r * pitch + c / 2) = packed;
  const int tiles = tiles_per_row(FMT, cols), tj = c / (4 * kBlock<FMT>);
  if (lane % (4 * LB) == 0 && tj < tiles)
    *reinterpret_cast<uint32_t*>(scales + scale_word_offset(r, tj, tiles)) = word;
}

template <typename T>
__device__ __forceinline__ float load_f32(const T* p) {
  if constexpr (sizeof(T) == 2)
    return __bfloat162float(*p);
  else
    return *p;
}
template <typename T>
__device__ __forceinline__ void store_f32(T* p, float v) {
  if constexpr (sizeof(T) == 2)
    *p = __float2bfloat16_rn(v);
  else
    *p = v;
}

// Eight consecutive elements from column c (zero from column cols on).  vec: the
// row's address and c allow 16-byte loads.
template <typename T>
__device__ __forceinline__ void load8(const T* row, int c, int cols, bool vec, float (&v)[8]) {
  if (vec && c + 8 <= cols) {
    if constexpr (sizeof(T) == 2) {
      const uint4 u = *reinterpret_cast<const uint4*>(row + c);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
      const float4 a = *reinterpret_cast<const float4*>(row + c);
      const float4 b = *reinterpret_cast<const float4*>(row + c + 4);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? load_f32(row + c + i) : 0.0f;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* row, int c, int cols, bool vec, const float (&v)[8]) {
  if (vec && c + 8 <= cols) {
    if constexpr (sizeof(T) == 2) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(row + c) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      *reinterpret_cast<float4*>(row + c) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(row + c + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) store_f32(row + c + i, v[i]);
  }
}

// Whether rows of T at p, ld elements apart, allow 16-byte accesses at columns that
// are multiples of 8.
template <typename T>
inline bool rows_vec(const void* p, long long ld) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * (long long)sizeof(T)) % 16 == 0;
}

// GELU, x Phi(x).  Phi(-|x|) = 1/2 (a1 u + .. + a5 u^5) exp(-x^2 / 2) with
// u = 1 / (1 + p |x| / sqrt 2): Abramowitz and Stegun 7.1.26, within 0.75e-7 of Phi
// (the product's own rounding is larger), one reciprocal and one exponential.
__device__ __forceinline__ float gelu(float x) {
  const float u = __fdividef(1.0f, fmaf(0.3275911f * 0.70710678f, fabsf(x), 1.0f));
  float q = fmaf(1.061405429f, u, -1.453152027f);
  q = fmaf(q, u, 1.421413741f);
  q = fmaf(q, u, -0.284496736f);
  q = fmaf(q, u, 0.254829592f);
  q = 0.5f * q * u * __expf(-0.5f * x * x);
  return x * (x < 0.0f ? q : 1.0f - q);
}

// The epilogue's activation over N values.  SiLU: x / (1 + exp(-x)) (exp overflows to
// infinity for very negative x, the quotient is then -0).  Comparisons keep a NaN.
template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
  if (act == CONV_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i];
  } else if (act == CONV_ACT_RELU6) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = v[i] < 0.0f ? 0.0f : (v[i] > 6.0f ? 6.0f : v[i]);
  } else if (act == CONV_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = gelu(v[i]);
  } else if (act == CONV_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __fdividef(v[i], 1.0f + __expf(-v[i]));
  }
}

}  // namespace fp4
}  // namespace gb
