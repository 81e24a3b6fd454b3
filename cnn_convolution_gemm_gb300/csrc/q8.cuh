// Device code shared by the kernels that make or read 8-bit matrices with scales (E4M3
// values or whole numbers; the formats and their layout in memory are defined in gbconv.h).
#pragma once

#include "fp4.cuh"

namespace gb {
namespace q8 {

constexpr int GROUP = 128;  // columns that share a scale, where a row has several

// Bytes between rows of codes, and scales of a row.
__host__ __device__ constexpr long long code_pitch(int cols) {
  return 16LL * ((cols + 15LL) / 16);
}
__host__ __device__ constexpr int scales_per_row(int group, int cols) {
  return group ? (int)((cols + (long long)GROUP - 1) / GROUP) : 1;
}

// Four values, each the nearest code of v * r.
template <int FMT>
__device__ __forceinline__ uint32_t pack4(const float* v, float r) {
  uint32_t w;
  if constexpr (FMT == CONV_Q8_E4M3) {
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(w)
        : "f"(v[0] * r), "f"(v[1] * r), "f"(v[2] * r), "f"(v[3] * r));
  } else {
    // 1.5 * 2^23 has a unit of 1: the sum's low byte is the whole number
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(fmaf(v[i], r, 12582912.0f));
    w = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  }
  return w;
}

// The magnitude of a code, and the values of four.
template <int FMT>
__device__ __forceinline__ float magnitude(uint32_t byte) {
  if constexpr (FMT == CONV_Q8_E4M3) return fp4::from_e4m3(byte & 0x7Fu);
  return (float)abs((int)(int8_t)byte);
}
template <int FMT>
__device__ __forceinline__ void unpack4(uint32_t w, float* v) {
  if constexpr (FMT == CONV_Q8_E4M3) {
    asm("{\n\t.reg .b16 lo, hi, a0, a1, a2, a3;\n\t.reg .b32 h0, h1;\n\t"
        "mov.b32 {lo, hi}, %4;\n\t"
        "cvt.rn.f16x2.e4m3x2 h0, lo;\n\tcvt.rn.f16x2.e4m3x2 h1, hi;\n\t"
        "mov.b32 {a0, a1}, h0;\n\tmov.b32 {a2, a3}, h1;\n\t"
        "cvt.f32.f16 %0, a0;\n\tcvt.f32.f16 %1, a1;\n\t"
        "cvt.f32.f16 %2, a2;\n\tcvt.f32.f16 %3, a3;\n\t}"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
        : "r"(w));
  } else {
    // 2^23 + (code + 128), less 2^23 + 128
    const uint32_t u = w ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 | i)) - 8388736.0f;
  }
}

// Which of two neighbouring codes (bytes of w and up, up the larger magnitude) are the nearest
// to v / s, ties to the even one: the sign of |v| - m s decides, m between them; one fma, so it
// is the exact one.  Seldom taken.
template <int FMT>
__device__ __forceinline__ uint32_t settle(const float* v, float s, uint32_t w, uint32_t up) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = (w >> (8 * i)) & 255u, b = (up >> (8 * i)) & 255u;
    if (a == b) continue;
    const float m = 0.5f * (magnitude<FMT>(a) + magnitude<FMT>(b));
    const float e = fmaf(-m, s, fabsf(v[i]));
    if (e > 0.0f || (e == 0.0f && (a & 1u))) w ^= (a ^ b) << (8 * i);
  }
  return w;
}

// The scale of a row or group from its largest magnitude, and the codes under it.
template <int FMT>
struct Scale {
  float s;           // NaN: the row or group is not finite
  float r_lo, r_hi;  // just below and just above 1 / s

  __device__ __forceinline__ explicit Scale(float top) {
    constexpr float T = FMT == CONV_Q8_E4M3 ? 448.0f : 127.0f;
    const bool bad = ((__float_as_uint(top) >> 23) & 255u) == 255u;
    s = bad ? __int_as_float(0x7FFFFFFF)
            : fmaxf(fp4::quotient(top, T, 1.0f / T, 3.4e38f), 0x1p-100f);
    // rcp_approx is within 2^-23, each rounding within 2^-24
    const float r = bad ? 0.0f : fp4::rcp_approx(s);
    r_lo = r * (1.0f - 0x1p-21f);
    r_hi = r * (1.0f + 0x1p-21f);
  }

  // Four codes, exact: where both sides of 1 / s give the same code it is x / s's too.
  __device__ __forceinline__ uint32_t codes4(const float* v) const {
    uint32_t w = pack4<FMT>(v, r_lo);
    const uint32_t up = pack4<FMT>(v, r_hi);
    if (w != up) w = settle<FMT>(v, s, w, up);
    return r_hi == 0.0f ? 0u : w;
  }
  __device__ __forceinline__ uint4 codes16(const float (&v)[16]) const {
    return make_uint4(codes4(v), codes4(v + 4), codes4(v + 8), codes4(v + 12));
  }
};

__device__ __forceinline__ float top16(const float (&v)[16], float top = 0.0f) {
#pragma unroll
  for (int i = 0; i < 16; i += 2) top = fp4::max_abs(top, v[i], v[i + 1]);
  return top;
}

// A lane's 16 consecutive columns of a row from column c on; LANES neighbours share a scale:
// the eight of a group of 128 columns, or all of a row of up to 16 LANES columns.  All lanes
// call it; valid: whether the row exists.
template <int FMT, int LANES = GROUP / 16>
__device__ __forceinline__ void store_grouped16(const float (&v)[16], bool valid, long long r,
                                                int c, int cols, uint8_t* codes, float* scales) {
  float top = top16(v);
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1)
    top = fp4::max_abs(top, top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  const Scale<FMT> s(top);
  const uint4 w = s.codes16(v);
  if (!valid || c >= cols) return;
  *reinterpret_cast<uint4*>(codes + r * code_pitch(cols) + c) = w;
  constexpr int SHARE = 16 * LANES;
  if (c % SHARE == 0) scales[r * ((cols + SHARE - 1) / SHARE) + c / SHARE] = s.s;
}

}  // namespace q8
}  // namespace gb
