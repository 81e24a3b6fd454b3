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

// The values of the eight codes in w.
__device__ __forceinline__ void unpack8_e2m1(uint32_t w, float (&v)[8]) {
  asm("{\n\t.reg .b8 t0, t1, t2, t3;\n\t.reg .b32 h0, h1, h2, h3;\n\t"
      ".reg .b16 a0, a1, a2, a3, a4, a5, a6, a7;\n\t"
      "mov.b32 {t0, t1, t2, t3}, %8;\n\t"
      "cvt.rn.f16x2.e2m1x2 h0, t0;\n\tcvt.rn.f16x2.e2m1x2 h1, t1;\n\t"
      "cvt.rn.f16x2.e2m1x2 h2, t2;\n\tcvt.rn.f16x2.e2m1x2 h3, t3;\n\t"
      "mov.b32 {a0, a1}, h0;\n\tmov.b32 {a2, a3}, h1;\n\t"
      "mov.b32 {a4, a5}, h2;\n\tmov.b32 {a6, a7}, h3;\n\t"
      "cvt.f32.f16 %0, a0;\n\tcvt.f32.f16 %1, a1;\n\tcvt.f32.f16 %2, a2;\n\t"
      "cvt.f32.f16 %3, a3;\n\tcvt.f32.f16 %4, a4;\n\tcvt.f32.f16 %5, a5;\n\t"
      "cvt.f32.f16 %6, a6;\n\tcvt.f32.f16 %7, a7;\n\t}"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7])
      : "r"(w));
}

// The E4M3 byte nearest to v (>= 0; above 448: 448), and the value of such a byte.
__device__ __forceinline__ uint32_t to_e4m3(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
  return r & 0xFFu;
}
__device__ __forceinline__ float from_e4m3(uint32_t b) {
  float v;
  asm("{\n\t.reg .b32 h;\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.f16x2.e4m3x2 h, %1;\n\t"
      "mov.b32 {lo, hi}, h;\n\t"
      "cvt.f32.f16 %0, lo;\n\t}"
      : "=f"(v)
      : "h"((uint16_t)b));
  return v;
}

// Two fp32 values in one register pair: a packed operation is one instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// About 2^-23 relative; 1 / 0 = inf, 1 / inf = 0.
__device__ __forceinline__ float rcp_approx(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float ex2_approx(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// max(|a|, |b|, |c|); a NaN stays.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// max and min of two values; a NaN stays.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// 1 for v > 0 (v itself a normal number), else 0.
__device__ __forceinline__ float positive(float v) {
  float r;
  asm("mul.rn.sat.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(3e38f));
  return r;
}
// v cut to [-lim, lim], lim >= 0
__device__ __forceinline__ float clamp_abs(float v, float lim) {
  float r;
  asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(lim));
  return r;
}

// A tensor scale g with what NV blocks need of it: t6 = 6 g and r6 = 1 / t6, rounded.
struct TensorScale {
  float g, t6, r6;
};
inline TensorScale tensor_scale(float g) {
  const float t6 = 6.0f * g;
  return {g, t6, 1.0f / t6};
}

// v / t rounded to nearest, from r = 1 / t: q0 = v r and the exact remainder
// v - q0 t (one fma) correct each other (Markstein's correction), so that a quotient
// that is a tie of E2M1 or E4M3 arrives there exactly.  Quotients above most come out
// as some value above most (v r may overflow).
__device__ __forceinline__ float quotient(float v, float t, float r, float most) {
  const float q0 = clamp_abs(v * r, most);
  return __fmaf_rn(__fmaf_rn(-q0, t, v), r, q0);
}

// The scale byte of a block from its largest magnitude, and its codes.
template <int FMT>
struct BlockScale {
  uint32_t byte;
  float t, r;  // MX: r alone, a power of two; NV: the divisor s * g and its reciprocal

  __device__ __forceinline__ BlockScale(float amax, const TensorScale& ts) {
    const uint32_t e = (__float_as_uint(amax) >> 23) & 255u;  // amax >= 0 or a NaN
    const bool bad = e == 255u;
    if (FMT == CONV_FP4_MX) {
      // floor(log2 amax) = e - 127 for normal numbers; e <= 2 and subnormals: 2^-127
      byte = bad ? 255u : (e > 2u ? e - 2u : 0u);
      r = bad ? 0.0f : __uint_as_float((254u - byte) << 23);  // 2^(127 - byte)
    } else {
      byte = bad ? 0x7Fu : to_e4m3(quotient(amax, ts.t6, ts.r6, 1024.0f));
      t = from_e4m3(byte) * ts.g;
      // 1 / t, one Newton step from the approximation
      const float r0 = rcp_approx(t);
      r = __fmaf_rn(__fmaf_rn(-t, r0, 1.0f), r0, r0);
      if (bad || byte == 0u) t = r = 0.0f;  // all codes 0
    }
  }
  // codes of eight elements of the block
  __device__ __forceinline__ uint32_t codes(const float (&v)[8]) const {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const uint64_t q0 = mul2(pack2(v[i], v[i + 1]), pack2(r, r));
      unpack2(q0, q[i], q[i + 1]);
      if (FMT == CONV_FP4_NV) {
        // quotient() on pairs
        q[i] = clamp_abs(q[i], 8.0f);
        q[i + 1] = clamp_abs(q[i + 1], 8.0f);
        const uint64_t c = pack2(q[i], q[i + 1]);
        const uint64_t e = fma2(pack2(-q[i], -q[i + 1]), pack2(t, t), pack2(v[i], v[i + 1]));
        unpack2(fma2(e, pack2(r, r), c), q[i], q[i + 1]);
      }
    }
    const uint32_t packed = pack8_e2m1(q);
    return r == 0.0f ? 0u : packed;  // Inf * 0 in a block that is not finite
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

// A lane's 16 consecutive elements of a row: their codes, and the scale word of their
// tile (complete in each of the tile's lanes).  MX: two lanes share a block and eight a
// scale tile; NV: one and four; all lanes call it.
template <int FMT>
__device__ __forceinline__ void quantize16(const float (&v)[16], const TensorScale& ts,
                                           uint2& codes, uint32_t& word) {
  constexpr int LB = kBlock<FMT> / 16;  // lanes per block
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; i += 2) top = max_abs(top, v[i], v[i + 1]);
  if (LB == 2) top = max_abs(top, top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  const BlockScale<FMT> s(top, ts);
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo[i] = v[i];
    hi[i] = v[8 + i];
  }
  codes = make_uint2(s.codes(lo), s.codes(hi));
  word = s.byte << (8 * (((threadIdx.x & 31) / LB) & 3));
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, LB);
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2 * LB);
}

// Stores such a lane's part of row r, from column c.
template <int FMT>
__device__ __forceinline__ void store_quantized16(const uint2& packed, uint32_t word, long long r,
                                                  int c, int cols, uint8_t* __restrict__ codes,
                                                  uint8_t* __restrict__ scales) {
  const long long pitch = code_pitch(cols);
  if (c < 2 * pitch) *reinterpret_cast<uint2*>(codes + r * pitch + c / 2) = packed;
  const int tiles = tiles_per_row(FMT, cols), tj = c / (4 * kBlock<FMT>);
  if (c % (4 * kBlock<FMT>) == 0 && tj < tiles)
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

// 32 and 16 bytes of global memory, past L1 (read once; L1 is left to what is reused).
struct alignas(32) Bytes32 {
  uint32_t w[8];
};
__device__ __forceinline__ Bytes32 load_stream32(const void* p) {
  Bytes32 r;
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]),
                 "=r"(r.w[5]), "=r"(r.w[6]), "=r"(r.w[7])
               : "l"(p));
  return r;
}
__device__ __forceinline__ void store32(void* p, const Bytes32& v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v.w[0]),
               "r"(v.w[1]), "r"(v.w[2]), "r"(v.w[3]), "r"(v.w[4]), "r"(v.w[5]), "r"(v.w[6]),
               "r"(v.w[7])
               : "memory");
}

// 16 consecutive elements of a row as they lie in memory.
template <typename T>
struct Raw16 {
  static constexpr int N = sizeof(T) / 2;  // 32-byte pieces
  Bytes32 b[N];

  // Elements from column c (zero from column cols on).  vec: the row allows 32-byte
  // accesses at columns that are multiples of 16.
  __device__ __forceinline__ void load(const T* row, int c, int cols, bool vec) {
    if (vec && c + 16 <= cols) {
#pragma unroll
      for (int i = 0; i < N; ++i) b[i] = load_stream32(row + c + i * (16 / N));
    } else {
#pragma unroll
      for (int i = 0; i < 8 * N; ++i) {
        uint32_t w = 0;
        if constexpr (sizeof(T) == 2) {
          const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
          if (c + 2 * i < cols) w = p[c + 2 * i];
          if (c + 2 * i + 1 < cols) w |= (uint32_t)p[c + 2 * i + 1] << 16;
        } else {
          if (c + i < cols) w = reinterpret_cast<const uint32_t*>(row)[c + i];
        }
        b[i / 8].w[i % 8] = w;
      }
    }
  }
  __device__ __forceinline__ void get(float (&v)[16]) const {
#pragma unroll
    for (int i = 0; i < 8 * N; ++i) {
      const uint32_t w = b[i / 8].w[i % 8];
      if constexpr (sizeof(T) == 2) {
        v[2 * i] = __uint_as_float(w << 16);
        v[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
      } else {
        v[i] = __uint_as_float(w);
      }
    }
  }
};

// 16 bytes of global memory that a neighbouring lane may load too.
__device__ __forceinline__ uint4 load16_cached(const void* p) {
  uint4 r;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// Raw16 of rows at any alignment: the 16-byte words that hold the elements, and how far
// into the first of them they start.  Single elements at the tensor's two ends, so that
// no word reaches outside it.
template <typename T>
struct RawAny16 {
  static constexpr int N = sizeof(T) / 2, WORDS = 8 * N;
  uint32_t w[WORDS + 4];
  uint32_t shift;  // bytes

  // first, last: the tensor's first and last rows (at least 16 columns, rows no closer)
  __device__ __forceinline__ void load(const T* row, int c, int cols, bool first, bool last) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + c);
    // a word starts up to 14 bytes before the elements and ends up to 14 bytes after them:
    // in this row, or in the one before or after
    if (c + 16 <= cols && (c > 0 || !first) && (c + 24 <= cols || !last)) {
      shift = at & 15;
      const char* const p = reinterpret_cast<const char*>(at - shift);
#pragma unroll
      for (int i = 0; i <= 2 * N; ++i) {
        // the last word holds nothing where the elements start on a word
        const uint4 v = i < 2 * N || shift ? load16_cached(p + 16 * i) : make_uint4(0, 0, 0, 0);
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
      }
    } else {
      shift = 0;
      Raw16<T> raw;
      raw.load(row, c, cols, false);
#pragma unroll
      for (int i = 0; i < WORDS; ++i) w[i] = raw.b[i / 8].w[i % 8];
#pragma unroll
      for (int i = WORDS; i < WORDS + 4; ++i) w[i] = 0;
    }
  }
  __device__ __forceinline__ void get(float (&v)[16]) const {
    uint32_t a[WORDS + 2], b[WORDS + 1];
#pragma unroll
    for (int i = 0; i < WORDS + 2; ++i) a[i] = shift & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < WORDS + 1; ++i) b[i] = shift & 4 ? a[i + 1] : a[i];
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
      if constexpr (sizeof(T) == 2) {
        const uint32_t h = __funnelshift_r(b[i], b[i + 1], (shift & 2) * 8);
        v[2 * i] = __uint_as_float(h << 16);
        v[2 * i + 1] = __uint_as_float(h & 0xFFFF0000u);
      } else {
        v[i] = __uint_as_float(b[i]);
      }
    }
  }
};

// 16 consecutive columns of a row that allows 32-byte accesses.
template <typename T>
__device__ __forceinline__ void store16(T* row, int c, int cols, const float (&v)[16]) {
  if (c + 16 <= cols) {
    constexpr int N = sizeof(T) / 2;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      Bytes32 b;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr (sizeof(T) == 2) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
          b.w[k] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          b.w[k] = __float_as_uint(v[8 * i + k]);
        }
      }
      store32(row + c + i * (16 / N), b);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (c + i < cols) store_f32(row + c + i, v[i]);
  }
}

// Stores consecutive columns of a row at any alignment, from column c0, 16 to a lane (v), up
// to column cols.  lane, lanes: which of the lanes that share the row (a warp, or a part of
// it).  A lane hands the elements that lie in its neighbour's 16-byte words on to it, and
// stores the words that its own elements and the ones it got fill; single elements where
// the lanes' columns begin and end inside a word.  All lanes of the warp call it; cols <= c0
// stores nothing.
template <typename T>
__device__ __forceinline__ void store_warp_any16(T* row, int c0, int cols, const float (&v)[16],
                                                 int lane, int lanes) {
  constexpr int WORDS = 4 * sizeof(T), PER = 16 / sizeof(T);  // 32-bit words, elements of 16 bytes
  const int c = c0 + lane * 16;
  const int end = c0 + 16 * lanes < cols ? c0 + 16 * lanes : cols;
  const uint32_t shift = reinterpret_cast<uintptr_t>(row + c0) & 15;
  const int ahead = (int)(shift / sizeof(T));  // elements in front of the first in its word
  uint32_t a[WORDS + 4];
#pragma unroll
  for (int i = 0; i < WORDS; ++i) {
    if constexpr (sizeof(T) == 2) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      a[4 + i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      a[4 + i] = __float_as_uint(v[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = __shfl_up_sync(0xFFFFFFFFu, a[WORDS + i], 1);
  // the words from 16 - shift bytes on
  const uint32_t from = 16 - shift;
  uint32_t b[WORDS + 2], d[WORDS + 1];
  if (from & 16) {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) a[i] = a[i + 4];
  }
#pragma unroll
  for (int i = 0; i < WORDS + 2; ++i) b[i] = from & 8 ? a[i + 2] : a[i];
#pragma unroll
  for (int i = 0; i < WORDS + 1; ++i) d[i] = from & 4 ? b[i + 1] : b[i];
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) d[i] = __funnelshift_r(d[i], d[i + 1], (from & 2) * 8);
  }
#pragma unroll
  for (int k = 0; k < WORDS / 4; ++k) {
    const int first = c - ahead + k * PER;
    if (first >= c0 && first + PER <= end) {
      *reinterpret_cast<uint4*>(row + first) =
          make_uint4(d[4 * k], d[4 * k + 1], d[4 * k + 2], d[4 * k + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (first + i < c0 || first + i >= end) continue;
        if constexpr (sizeof(T) == 2)
          reinterpret_cast<uint16_t*>(row)[first + i] =
              (uint16_t)(d[4 * k + i / 2] >> (16 * (i & 1)));
        else
          reinterpret_cast<uint32_t*>(row)[first + i] = d[4 * k + i];
      }
    }
  }
  if (lane == lanes - 1) {  // what would have been handed on
#pragma unroll
    for (int i = 16 - PER; i < 16; ++i)
      if (i >= 16 - ahead && c + i < cols) store_f32(row + c + i, v[i]);
  }
}

// Whether rows of T at p, ld elements apart, allow accesses of so many bytes at columns
// that are multiples of them.
template <typename T>
inline bool rows_vec(const void* p, long long ld, int bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && (ld * (long long)sizeof(T)) % bytes == 0;
}

// GELU of two values, x Phi(x) = max(x, 0) + |x| q with q = -Phi(-|x|) = -u Q(u) exp(-x^2 / 2),
// u = 1 / (1 + p |x|) and a polynomial Q.
// FP32, for outputs of 32 bits: u Q(u) = Phi(-a) exp(a^2 / 2) with p = 0.305 makes Q smooth on
// (0, 1]; degree 7, with little cancellation (the magnitudes of its terms add up to 0.85, Q to
// 0.12 .. 0.5), is within 1e-7 of its value, fitted here for a up to 14.5 by least squares with
// Lawson's weights for the least maximum.  As evaluated within (x^2 + 14) 2^-23 of the result.
// Else degree 4, Abramowitz and Stegun 7.1.26, whose own error is 0.75e-7 of Phi; as evaluated
// x Phi(x) is within 4.2e-7, and relatively within 6e-5 above x = -3 and 2e-3 above -5 (bf16
// rounds by up to 4e-3).  20128 x 384 x 2304 to bf16 36.3 us, with the longer one 38.6.
template <bool FP32>
__device__ __forceinline__ void gelu2(float& x0, float& x1) {
  // q is 0 well below 64: an infinity must not meet it
  const float a0 = fminf(fabsf(x0), 64.0f), a1 = fminf(fabsf(x1), 64.0f);
  const uint64_t x = pack2(x0, x1), a = pack2(a0, a1);
  constexpr int D = FP32 ? 7 : 4;
  constexpr float P = FP32 ? 0.305f : 0.23164189f;  // 0.3275911 / sqrt 2
  constexpr float C7[8] = {-0.12164024f, -0.12245868f, -0.10347369f, -0.12084042f,
                           0.03762071f,  -0.18531495f, 0.15274611f,  -0.036638875f};
  constexpr float C4[5] = {-0.5f * 0.254829592f, 0.5f * 0.284496736f, -0.5f * 1.421413741f,
                           0.5f * 1.453152027f, -0.5f * 1.061405429f};
  float d0, d1, e0, e1;
  unpack2(fma2(a, pack2(P, P), pack2(1.0f, 1.0f)), d0, d1);
  const uint64_t u = pack2(rcp_approx(d0), rcp_approx(d1));
  const float top = FP32 ? C7[7] : C4[4];
  uint64_t q = pack2(top, top);
#pragma unroll
  for (int i = D - 1; i >= 0; --i) {
    const float c = FP32 ? C7[i] : C4[i < 5 ? i : 4];
    q = fma2(q, u, pack2(c, c));
  }
  const float k = -0.5f * 1.4426950408889634f;  // exp(-x^2 / 2) = 2^(k x^2)
  unpack2(mul2(mul2(x, pack2(k, k)), x), e0, e1);
  q = mul2(mul2(q, u), pack2(ex2_approx(e0), ex2_approx(e1)));
  // max(x, 0) as x * (x > 0), which is NaN for -inf
  unpack2(fma2(x, pack2(positive(x0), positive(x1)), mul2(a, q)), x0, x1);
}

// 1 / (1 + exp(-v)), 0 below about -87.  FP32: within 2^-21 of its value.  Else the rounding of
// v log2 e enters, and it is within (|v| + 8) 2^-23, as outputs of 16 and 4 bits need it.
template <bool FP32>
__device__ __forceinline__ float logistic(float v) {
  return rcp_approx(1.0f + (FP32 ? expf(-v) : ex2_approx(v * -1.4426950408889634f)));
}

// The epilogue's activation over N values.  FP32: for an fp32 output.  SiLU: x / (1 + exp(-x))
// (exp overflows to infinity for very negative x, the quotient is then -0).  Comparisons keep a
// NaN; GELU and SiLU of -inf are one (inf * 0).
template <bool FP32, int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
  if (act == CONV_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = max_nan(v[i], 0.0f);
  } else if (act == CONV_ACT_RELU6) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = min_nan(max_nan(v[i], 0.0f), 6.0f);
  } else if (act == CONV_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; i += 2) gelu2<FP32>(v[i], v[i + 1]);
  } else if (act == CONV_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= logistic<FP32>(v[i]);
  }
}

}  // namespace fp4
}  // namespace gb
