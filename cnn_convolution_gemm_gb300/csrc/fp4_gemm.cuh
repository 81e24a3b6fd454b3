// What the products of 4-bit matrices share: the k-step and the TMA maps of the operands.
#pragma once

#include "fp4.cuh"
#include "internal.h"

namespace gb {
namespace fp4 {

constexpr int BKB = 128;  // bytes of a row per k-step: 256 codes

// Rows that a load of a 128-row tile brings: 64 where no more are left of total, none past
// its end.  A box whose second 64 rows lie outside the matrix altogether is slow (33 .. 63
// x 4096 x 16384 10.5 us with boxes of 128 rows, 64 or more rows 7.0).
__host__ __device__ constexpr int box_rows(int row0, int total) {
  return total - row0 > 64 ? 128 : total - row0 > 0 ? 64 : 0;
}
// Whether the last tile of so many rows takes a 64-row box.
inline bool short_tail(int total) { return box_rows((total - 1) / 128 * 128, total) == 64; }

// [rows][pitch] bytes of codes in boxes of 128 bytes x box_rows
inline bool codes_map(CUtensorMap* map, const uint8_t* p, int rows, int cols, int box_rows) {
  cuuint64_t dims[2] = {(cuuint64_t)code_pitch(cols), (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)code_pitch(cols)};
  cuuint32_t box[2] = {BKB, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return gb_encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p), dims,
                         strides, box, estr, CU_TENSOR_MAP_SWIZZLE_128B) == CUDA_SUCCESS;
}
// scale tiles as [panels][tiles * 64] 8-byte elements, boxes of `atoms` tiles x `panels`
inline bool scales_map(CUtensorMap* map, const uint8_t* p, int fmt, int rows, int cols, int atoms,
                int box_panels) {
  const cuuint64_t w = (cuuint64_t)tiles_per_row(fmt, cols) * 64;
  cuuint64_t dims[2] = {w, (cuuint64_t)((rows + 127LL) / 128)};
  cuuint64_t strides[1] = {w * 8};
  cuuint32_t box[2] = {(cuuint32_t)(atoms * 64), (cuuint32_t)box_panels};
  cuuint32_t estr[2] = {1, 1};
  return gb_encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT64, 2, const_cast<uint8_t*>(p), dims,
                         strides, box, estr, CU_TENSOR_MAP_SWIZZLE_NONE) == CUDA_SUCCESS;
}

}  // namespace fp4
}  // namespace gb
