// How the kernels that quantise matrices, and those that read them back, walk over the rows.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>

#include "internal.h"

namespace gb {
namespace walk {

constexpr int THREADS = 256;
constexpr int ROWS = 2;  // rows whose loads a warp issues together

// A warp works on 512 columns of a row, 16 to a lane (32 bytes of bf16), and walks over
// rows.  Both directions should move bytes only: the loads of several rows are in flight
// per warp, and the instructions of an element are few.  Rows of up to 256 (128) columns
// share a warp two (four) at a time.  wx (a power of two up to 8) warps of a block lie
// side by side along a row, the others below one another.
struct Walk {
  int c;               // the lane's first column
  long long row, step; // the lane's first row, and rows between its rows
};
// NARROW: wx_log2 < 0, 1 << -wx_log2 rows to a warp
template <bool NARROW>
__device__ __forceinline__ Walk walk(int wx_log2) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Walk w;
  if constexpr (NARROW) {
    const int lanes_log2 = 5 + wx_log2;  // lanes of a row
    const int wy = (THREADS / 32) << -wx_log2;
    w.c = (lane & ((1 << lanes_log2) - 1)) * 16;
    w.row = (long long)blockIdx.y * wy + (warp << -wx_log2) + (lane >> lanes_log2);
    w.step = (long long)gridDim.y * wy;
    return w;
  }
  const int wy = (THREADS / 32) >> wx_log2;
  w.c = (((int)blockIdx.x << wx_log2) + (warp & ((1 << wx_log2) - 1))) * 512 +
        (threadIdx.x & 31) * 16;
  w.row = (long long)blockIdx.y * wy + (warp >> wx_log2);
  w.step = (long long)gridDim.y * wy;
  return w;
}

// Grid of a walk over rows x cols: the columns covered once, as many rows at a time as
// fill the SMs (8 blocks each) with ROWS rows to a warp.
struct Shape {
  dim3 grid;
  int wx_log2;
};
inline Shape walk_shape(int rows, int cols) {
  Shape s;
  const int chunks = (int)gb_ceil_div_ll(cols, 512);
  s.wx_log2 = cols <= 128 ? -2 : cols <= 256 ? -1 : 0;
  while (s.wx_log2 >= 0 && s.wx_log2 < 3 && (1 << s.wx_log2) < chunks) ++s.wx_log2;
  const int wy = s.wx_log2 < 0 ? (THREADS / 32) << -s.wx_log2 : (THREADS / 32) >> s.wx_log2;
  const int gx = s.wx_log2 < 0 ? 1 : gb_ceil_div(chunks, 1 << s.wx_log2);
  const long long need = gb_ceil_div_ll(rows, ROWS * wy);
  const long long gy = std::min<long long>(need, std::max(1, gb_num_sms() * 8 / gx));
  s.grid = dim3((unsigned)gx, (unsigned)gy);
  return s;
}

// Launch that may set up while the kernel before it drains (it waits for that kernel's
// end before it touches global memory).
template <int BLOCK = THREADS, typename... P, typename... A>
cudaError_t launch_walk(void (*kern)(P...), dim3 grid, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(BLOCK);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  if (e == cudaSuccess) gb_count_launch();
  return e;
}

}  // namespace walk
}  // namespace gb
