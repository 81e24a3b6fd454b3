// Product of two microscaled 4-bit matrices, y = act(alpha X W^T + bias + residual),
// on the block-scaled tcgen05 MMAs.
//
// GEMM names here: M rows of X, N rows of W (the layer's outputs), KR the reduction.
// Persistent CTAs: warp 0 loads (TMA), warp 1 copies the block scales to TMEM and issues
// the MMAs (one elected lane), warps 4 and up run the epilogue.  A k-step is 256 elements:
// 128-byte rows of codes (128-byte swizzle) and 512-byte scale tiles.
//
// Bound: shared memory.  A k-step of a 256 x 256 tile over an SM pair takes 513 cycles of
// MMAs (K = 64 each, measured alone); its 35 KB of operands (MX; NV 38 KB) are written by
// the TMA and read by the MMAs and scale copies at 128 bytes a cycle together: 547 (594).
// An MMA with K = 96 would not change that, which is why there is none here.  Beside the
// loop a tile takes 900 to 4000 cycles (one accumulator of 256 columns, which the epilogue has
// to read first; staged stores through the same shared memory).  Measured, rows x inputs x
// outputs: 8192 x 16384 x 4096 139 to 143 us MX, 152 to 154 NV (7.7 to 7.9, 7.1 to 7.3
// PFLOP/s); after two seconds of it, at the 1.71 and 1.64 GHz of the power limit, 152 and 166.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "fp4.cuh"
#include "fp4_gemm.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace {
using namespace gb::fp4;

constexpr int BM = 128;
constexpr int SPLIT_MOST = 8;  // CTAs of a cluster

template <int FMT, int BN, bool PAIR, int YIO>
struct Cfg {
  static constexpr int CW = BN / 4;       // columns of an epilogue warp
  static constexpr int EPI_WARPS = 16;    // 4 lane quarters x 4 column ranges
  static constexpr int THREADS = 128 + 32 * EPI_WARPS;
  static constexpr int ATOMS = FMT == CONV_FP4_MX ? 2 : 4;  // scale tiles per panel and k-step
  static constexpr int PB = (BN + 127) / 128;               // 128-row panels of W
  static constexpr int BROWS = PAIR ? BN / 2 : BN;          // rows of W this CTA loads
  static_assert(BROWS == 128, "box_rows");
  static constexpr int A_BYTES = BM * BKB;
  static constexpr int B_BYTES = BROWS * BKB;
  static constexpr int SFA_BYTES = ATOMS * 512;
  static constexpr int SFB_BYTES = PB * ATOMS * 512;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES;
  static constexpr int STAGES = 5;
  static constexpr int NACC = 2 * BN <= 256 ? 2 : 1;
  // scale columns of a stage, in a slot of its own per stage: a slot is written again
  // only after the MMAs that read it have committed the stage
  static constexpr int SF_COLS = ATOMS * 4 * (1 + PB);
  // of each epilogue warp: a staging buffer; 32 biases
  static constexpr int BUF = YIO == CONV_FP4_IO_CODES ? 0 : 2048;
  static constexpr int EPI_BYTES = EPI_WARPS * (BUF + 128);
  static constexpr int SMEM = STAGES * STAGE_BYTES + EPI_BYTES + 256 + 1024;
  static_assert(NACC * BN + STAGES * SF_COLS <= 512, "TMEM");
  static_assert(SMEM <= 232448, "shared memory");
};

struct GemmParams {
  int M, N, ksteps, kmmas_last;  // 64-element MMAs of the last k-step
  int m_tiles, n_tiles;          // PAIR: m_tiles counts 256-row units
  int split;                     // SPLIT: CTAs of a cluster
  int act, vec_y, vec_r;         // rows of y for the TMA (4-bit y: for 32-byte stores), of the
                                 // residual for 16-byte loads
  float alpha;
  TensorScale y_scale;
  const float* bias;
  const void* res;
  void* y;
  uint8_t* ys;
  long long ldr, ldy;
  int* err;
  unsigned long long wait_ns;
};

// ---- epilogue: a lane holds a row's fp32 accumulators ----------------------------------
//
// Rows of the output (and of the residual) pass through a staging buffer of the warp: 32
// rows of 64 bytes (COLS elements), their 16-byte pieces in the TMA's 64-byte swizzle, so
// that a quarter-warp's accesses hit all banks once, by row and by piece alike.  Where
// the output's rows allow it the TMA stores the buffer (and drops what lies outside):
// copied by the warp, 64 bytes a row, L1 was the bound (8192 x 256 x 4096: 73 % busy).

template <typename T>
struct Block {
  static constexpr int ES = sizeof(T);
  static constexpr int COLS = 64 / ES;

  static __device__ __forceinline__ uint8_t* at(uint8_t* buf, int row, int piece) {
    return buf + row * 64 + ((piece ^ ((row >> 1) & 3)) << 4);
  }
  static __device__ __forceinline__ T* elem(uint8_t* buf, int row, int col) {
    return reinterpret_cast<T*>(at(buf, row, col * ES / 16) + col * ES % 16);
  }
  // A block of global memory (rows < rows, columns < cols) into registers, and from
  // there into the buffer.  vec: four lanes to a row, 16 bytes each; else an element at a
  // time: a lane takes a column (bf16: all rows, two to a register; fp32: half the rows).
  static __device__ __forceinline__ void fetch(uint32_t (&r)[16], const T* g, long long ld,
                                               int rows, int cols, bool vec) {
    const int lane = threadIdx.x & 31;
    if (vec && cols >= COLS) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = i * 8 + lane / 4;
        uint4 u = make_uint4(0, 0, 0, 0);
        if (row < rows) u = *reinterpret_cast<const uint4*>(g + row * ld + lane % 4 * (16 / ES));
        r[4 * i] = u.x;
        r[4 * i + 1] = u.y;
        r[4 * i + 2] = u.z;
        r[4 * i + 3] = u.w;
      }
    } else {
      const int col = lane % COLS, row0 = lane / COLS * 16;
      const bool in = col < cols;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        r[i] = 0;
        if constexpr (ES == 2) {
          const uint16_t* const h = reinterpret_cast<const uint16_t*>(g) + col;
          if (in && 2 * i < rows) r[i] = h[2 * i * ld];
          if (in && 2 * i + 1 < rows) r[i] |= (uint32_t)h[(2 * i + 1) * ld] << 16;
        } else {
          if (in && row0 + i < rows)
            r[i] = reinterpret_cast<const uint32_t*>(g)[(row0 + i) * ld + col];
        }
      }
    }
  }
  static __device__ __forceinline__ void put(uint8_t* buf, const uint32_t (&r)[16], int cols,
                                             bool vec) {
    const int lane = threadIdx.x & 31;
    if (vec && cols >= COLS) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(at(buf, i * 8 + lane / 4, lane % 4)) =
            make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
    } else {
      const int col = lane % COLS, row0 = lane / COLS * 16;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if constexpr (ES == 2) {
          *reinterpret_cast<uint16_t*>(elem(buf, 2 * i, col)) = (uint16_t)r[i];
          *reinterpret_cast<uint16_t*>(elem(buf, 2 * i + 1, col)) = (uint16_t)(r[i] >> 16);
        } else {
          *reinterpret_cast<uint32_t*>(elem(buf, row0 + i, col)) = r[i];
        }
      }
    }
  }
};

// v (acc * alpha + bias) of rows m0.. and columns n0..: residual, activation, store (by
// the TMA: committed, and the buffer waited for before it is written again).
// pre: the residual, fetched ahead; refill() fetches what the warp needs next.
template <typename T, typename F>
__device__ __forceinline__ void finish_float(const GemmParams& p, const CUtensorMap* tm_y,
                                             float (&v)[Block<T>::COLS], uint8_t* buf, int m0,
                                             int n0, const uint32_t (&pre)[16], F refill) {
  using B = Block<T>;
  const int lane = threadIdx.x & 31;
  const int rows = min(32, p.M - m0), cols = min(B::COLS, p.N - n0);
  if (p.vec_y) {  // the buffer's last store has read it
    if (lane == 0) gb::bulk_wait_read<0>();
    __syncwarp();
  }
  if (p.res) {
    B::put(buf, pre, cols, p.vec_r);
    refill();
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 u = *reinterpret_cast<const uint4*>(B::at(buf, lane, i));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (B::ES == 2) {
          v[i * 8 + 2 * k] += __uint_as_float(w[k] << 16);
          v[i * 8 + 2 * k + 1] += __uint_as_float(w[k] & 0xFFFF0000u);
        } else {
          v[i * 4 + k] += __uint_as_float(w[k]);
        }
      }
    }
    __syncwarp();
  }
  activate<B::ES == 4>(v, p.act);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (B::ES == 2) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[i * 8 + 2 * k], v[i * 8 + 2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        w[k] = __float_as_uint(v[i * 4 + k]);
      }
    }
    *reinterpret_cast<uint4*>(B::at(buf, lane, i)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (p.vec_y) {
    gb::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      gb::tma_store_2d(tm_y, buf, n0, m0);
      gb::bulk_commit();
    }
  } else {
    __syncwarp();
    T* y = static_cast<T*>(p.y) + (long long)m0 * p.ldy + n0;
    if (lane < cols) {
#pragma unroll 4
      for (int r = 0; r < rows; ++r) y[r * p.ldy + lane] = *B::elem(buf, r, lane);
    }
    __syncwarp();
  }
}

// 32 columns of the lane's row (one MX block or two NV blocks): codes and scale bytes.
// cols: how many of the columns exist.
template <int FMT>
__device__ __forceinline__ void quantize32(const TensorScale& ts, float (&v)[32], int cols,
                                           uint32_t (&code)[4], uint32_t& bytes) {
  if (cols < 32) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i >= cols) v[i] = 0.0f;
  }
  constexpr int B = kBlock<FMT>;
  bytes = 0;
#pragma unroll
  for (int k = 0; k < 32 / B; ++k) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < B; i += 2) top = max_abs(top, v[k * B + i], v[k * B + i + 1]);
    const BlockScale<FMT> s(top, ts);
    bytes |= s.byte << (8 * k);
#pragma unroll
    for (int i = 0; i < B / 8; ++i) {
      float e[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) e[t] = v[k * B + i * 8 + t];
      code[k * (B / 8) + i] = s.codes(e);
    }
  }
}

// Stores such codes of row m, W columns from n0 on (32, or 64: whole 32-byte sectors), and
// the scales.
template <int FMT, int W>
__device__ __forceinline__ void store_codes(const GemmParams& p, long long m, int n0,
                                            const uint32_t (&code)[W / 8], uint32_t bytes) {
  constexpr int B = kBlock<FMT>;
  const long long pitch = code_pitch(p.N);
  const int tiles = tiles_per_row(FMT, p.N);
  uint8_t* const to = static_cast<uint8_t*>(p.y) + m * pitch + n0 / 2;
  // codes start and their rows lie on multiples of 16 bytes, not always of 32
  if (W == 64 && p.vec_y && n0 + 32 < p.N) {
    Bytes32 b;
#pragma unroll
    for (int i = 0; i < 8; ++i) b.w[i] = code[i % (W / 8)];
    store32(to, b);
  } else {
#pragma unroll
    for (int i = 0; i < W / 32; ++i)
      if (n0 + 32 * i < p.N)
        *reinterpret_cast<uint4*>(to + 16 * i) =
            make_uint4(code[4 * i], code[4 * i + 1], code[4 * i + 2], code[4 * i + 3]);
  }
  const int b0 = n0 / B;
  uint8_t* word = p.ys + scale_word_offset(m, b0 >> 2, tiles) + (b0 & 3);
  if constexpr (W / B == 4)
    *reinterpret_cast<uint32_t*>(word) = bytes;
  else if constexpr (W / B == 2)
    *reinterpret_cast<uint16_t*>(word) = (uint16_t)bytes;
  else
    *word = (uint8_t)bytes;
  // padding blocks of the row's last tile
  if (n0 + W >= p.N)
    for (int b = (n0 + W) / B; (b >> 2) < tiles; ++b)
      p.ys[scale_word_offset(m, b >> 2, tiles) + (b & 3)] = 0;
}

// SPLIT (128 x 128 tiles): the CTAs of a cluster share one tile, each with a range of the
// reduction.  An epilogue warp's block of 32 x 32 belongs to one of them, which gets the
// others' partial sums through distributed shared memory (in the ring, whose last
// operands are read by then) and adds them in the order of the ranges.
template <int FMT, int BN, bool PAIR, int YIO, bool SPLIT>
__global__ void __launch_bounds__(Cfg<FMT, BN, PAIR, YIO>::THREADS, 1)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap tm_x,
                    const __grid_constant__ CUtensorMap tm_xs,
                    const __grid_constant__ CUtensorMap tm_w,
                    const __grid_constant__ CUtensorMap tm_ws,
                    const __grid_constant__ CUtensorMap tm_y,
                    const __grid_constant__ CUtensorMap tm_x64,
                    const __grid_constant__ CUtensorMap tm_w64, const GemmParams p) {
  using C = Cfg<FMT, BN, PAIR, YIO>;
  constexpr bool MX = FMT == CONV_FP4_MX;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + C::STAGES * C::A_BYTES;
  uint8_t* sFA = sB + C::STAGES * C::B_BYTES;
  uint8_t* sFB = sFA + C::STAGES * C::SFA_BYTES;
  uint8_t* sEpi = sFB + C::STAGES * C::SFB_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(sEpi + C::EPI_BYTES);
  uint64_t* empty = full + C::STAGES;
  uint64_t* tfull = empty + C::STAGES;
  uint64_t* tempty = tfull + C::NACC;
  uint64_t* mma_done = tempty + C::NACC;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);

  const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0);  // uniform
  const int lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? gb::cluster_ctarank() : 0u;
  const int part = SPLIT ? (int)gb::cluster_ctarank() : 0;
  const int unit0 = PAIR ? (int)(blockIdx.x >> 1)
                    : SPLIT ? (int)blockIdx.x / p.split : (int)blockIdx.x;
  const int ustep = PAIR ? (int)(gridDim.x >> 1)
                    : SPLIT ? p.m_tiles * p.n_tiles : (int)gridDim.x;
  // this CTA's k-steps
  const int k0 = SPLIT ? (int)((long long)p.ksteps * part / p.split) : 0;
  const int k1 = SPLIT ? (int)((long long)p.ksteps * (part + 1) / p.split) : p.ksteps;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      gb::mbar_init(&full[s], 1);
      gb::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < C::NACC; ++b) {
      gb::mbar_init(&tfull[b], 1);
      gb::mbar_init(&tempty[b], C::EPI_WARPS * (PAIR ? 2 : 1));  // one arrival per epilogue warp
    }
    gb::mbar_init(mma_done, 1);
    gb::fence_barrier_init();
    gb::tma_prefetch_desc(&tm_x);
    gb::tma_prefetch_desc(&tm_w);
    gb::tma_prefetch_desc(&tm_xs);
    gb::tma_prefetch_desc(&tm_ws);
    if (YIO != CONV_FP4_IO_CODES && p.vec_y) gb::tma_prefetch_desc(&tm_y);
  }
  if (warp == 0) {
    if constexpr (PAIR) {
      gb::tmem_alloc_pair(tmem_slot, 512);
      gb::tmem_relinquish_pair();
    } else {
      gb::tmem_alloc(tmem_slot, 512);
      gb::tmem_relinquish();
    }
  }
  gb::tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) gb::cluster_sync();
  gb::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  gb::allow_dependents();

  const int units = p.m_tiles * p.n_tiles;
  // 256 columns: the launch's registers, 640 x 96, as 128 x 40 + 512 x 104 (at most)
  if (warp < 4) {
    if constexpr (BN == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0) {
      // ---------------- TMA producer ----------------
      const bool one = gb::elect_one();
      int stage = 0;
      uint32_t phase = 0;
      long long issued = 0;
      bool ok = true;
      const uint32_t full_pair = PAIR ? gb::mapa_shared(gb::smem_u32(full), 0) : 0u;
      asm volatile("griddepcontrol.wait;" ::: "memory");
      for (int u = unit0; u < units && ok; u += ustep) {
        const int mt = (u / p.n_tiles) * (PAIR ? 2 : 1) + (int)rank, nt = u % p.n_tiles;
        const int brow = nt * BN + (PAIR ? (int)rank * C::BROWS : 0);
        // rows past the ends are not loaded: what the tile's memory holds there reaches
        // accumulators of rows and columns that nobody stores
        const int ar = box_rows(mt * BM, p.M), br = box_rows(brow, p.N);
        const CUtensorMap* const xmap = ar == 64 ? &tm_x64 : &tm_x;
        const CUtensorMap* const wmap = br == 64 ? &tm_w64 : &tm_w;
        uint32_t tx = (ar + br) * BKB + (ar ? C::SFA_BYTES : 0) + C::SFB_BYTES;
        if (PAIR)  // of both CTAs
          tx += (box_rows((mt + 1) * BM, p.M) + box_rows(brow + C::BROWS, p.N)) * BKB +
                ((mt + 1) * BM < p.M ? C::SFA_BYTES : 0) + C::SFB_BYTES;
        for (int it = k0; it < k1; ++it) {
          if (!gb::mbar_wait_bounded_warp(&empty[stage], phase ^ 1, p.wait_ns, p.err)) {
            ok = false;
            break;
          }
          if (one) {
            uint8_t* const a = sA + stage * C::A_BYTES;
            uint8_t* const b = sB + stage * C::B_BYTES;
            uint8_t* const fa = sFA + stage * C::SFA_BYTES;
            uint8_t* const fb = sFB + stage * C::SFB_BYTES;
            const int sc = it * (C::ATOMS * 64);  // scale tiles as 8-byte elements
            if constexpr (PAIR) {
              if (rank == 0) gb::mbar_arrive_expect_tx(&full[stage], tx);
              const uint32_t bar = full_pair + stage * 8;
              if (ar) gb::tma_load_2d_pair(a, xmap, bar, it * BKB, mt * BM);
              if (br) gb::tma_load_2d_pair(b, wmap, bar, it * BKB, brow);
              if (ar) gb::tma_load_2d_pair(fa, &tm_xs, bar, sc, mt);
              gb::tma_load_2d_pair(fb, &tm_ws, bar, sc, nt * BN / 128);
            } else {
              gb::mbar_arrive_expect_tx(&full[stage], tx);
              gb::tma_load_2d(a, xmap, &full[stage], it * BKB, mt * BM);
              gb::tma_load_2d(b, wmap, &full[stage], it * BKB, brow);
              gb::tma_load_2d(fa, &tm_xs, &full[stage], sc, mt);
              gb::tma_load_2d(fb, &tm_ws, &full[stage], sc, nt * BN / 128);
            }
          }
          __syncwarp();
          ++issued;
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // no copy into shared memory may be in flight at exit (pair: the even CTA's
      // barriers count both CTAs' bytes, so it drains for both)
      long long pending = issued < C::STAGES ? issued : C::STAGES;
      if (PAIR && rank != 0) pending = 0;
      for (long long i = 0; i < pending; ++i) {
        if (--stage < 0) {
          stage = C::STAGES - 1;
          phase ^= 1;
        }
        gb::mbar_wait_bounded_warp(&full[stage], phase, p.wait_ns, p.err);
      }
    } else if (warp == 1 && rank == 0) {
      // ---------------- scale copies and MMAs ----------------
      const bool one = gb::elect_one();
      constexpr int MM = PAIR ? 2 * BM : BM;
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int u = unit0; u < units && ok; u += ustep) {
        const uint32_t d = tmem + acc * BN;
        for (int it = k0; it < k1; ++it) {
          if (!gb::mbar_wait_bounded_warp(&full[stage], phase, p.wait_ns, p.err)) {
            ok = false;
            break;
          }
          gb::tc_fence_after();
          const uint32_t sfa = tmem + C::NACC * BN + stage * C::SF_COLS;
          const uint32_t sfb = sfa + C::ATOMS * 4;
          if (one) {
            const uint32_t fa = gb::smem_u32(sFA + stage * C::SFA_BYTES);
            const uint32_t fb = gb::smem_u32(sFB + stage * C::SFB_BYTES);
            // scale tiles (32 rows x 16 bytes): A's tile j at columns 4 j, B's panel q of
            // tile j at 4 (j PB + q), so that an MMA's B scales are consecutive
#pragma unroll
            for (int j = 0; j < C::ATOMS; ++j) {
              gb::tc_copy_scales<PAIR>(sfa + 4 * j, gb::noswz_kmajor_desc(fa + j * 512, 128, 128));
#pragma unroll
              for (int q = 0; q < C::PB; ++q)
                gb::tc_copy_scales<PAIR>(
                    sfb + 4 * (j * C::PB + q),
                    gb::noswz_kmajor_desc(fb + (q * C::ATOMS + j) * 512, 128, 128));
            }
          }
          __syncwarp();
          // the tile's accumulator is needed only now
          if (it == k0) {
            if (!gb::mbar_wait_bounded_warp(&tempty[acc], acc_phase ^ 1, p.wait_ns, p.err)) {
              ok = false;
              break;
            }
            gb::tc_fence_after();
          }
          if (one) {
            const uint64_t ad = gb::sw128_kmajor_desc(gb::smem_u32(sA + stage * C::A_BYTES));
            const uint64_t bd = gb::sw128_kmajor_desc(gb::smem_u32(sB + stage * C::B_BYTES));
            const int mmas = it + 1 < p.ksteps ? 4 : p.kmmas_last;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              // MX: a scale word (4 blocks of 32) serves two MMAs; NV: (4 of 16) one
              const int j = MX ? k / 2 : k;
              const uint32_t id = gb::idesc_fp4(MM, BN, MX, MX ? (k & 1) * 2 : 0);
              if (k < mmas)
                gb::tc_mma_fp4<MX, PAIR>(d, ad + k * 2, bd + k * 2, id, sfa + 4 * j,
                                         sfb + 4 * j * C::PB, it > k0 || k > 0 ? 1u : 0u);
            }
            if constexpr (PAIR)
              gb::tc_commit_pair_multicast(&empty[stage], 0x3);
            else
              gb::tc_commit(&empty[stage]);
          }
          __syncwarp();
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if (one) {
          if constexpr (PAIR)
            gb::tc_commit_pair_multicast(&tfull[acc], 0x3);
          else
            gb::tc_commit(&tfull[acc]);
        }
        __syncwarp();
        if (++acc == C::NACC) {
          acc = 0;
          acc_phase ^= 1;
        }
      }
      if (one) {
        if constexpr (PAIR)
          gb::tc_commit_pair_multicast(mma_done, 0x1);
        else
          gb::tc_commit(mma_done);
      }
      __syncwarp();
      gb::mbar_wait_bounded_warp(mma_done, 0, p.wait_ns, p.err);
    }
    if constexpr (SPLIT) {  // the epilogue's two barriers
      __syncwarp();
      gb::cluster_sync();
      gb::cluster_sync();
    }
  } else {
    if constexpr (BN == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    // ---------------- epilogue (warps 4 and up) ----------------
    // A warp owns 32 rows (the TMEM lane quarter it may access) and a quarter of the tile's
    // columns.  It takes its accumulators into registers and frees the TMEM
    // accumulator before it works on them: the next tile's MMAs wait for TMEM reads only.
    // (With half the warps, two per scheduler, it was idle 65 % of the time:
    // 8192 x 4096 x 16384 with GELU 197 us against 186.)
    using T = std::conditional_t<YIO == CONV_FP4_IO_BF16, __nv_bfloat16, float>;
    constexpr bool FLOAT = YIO != CONV_FP4_IO_CODES;
    constexpr int PC = FLOAT ? Block<T>::COLS : 32;  // columns of a pass
    constexpr int CW = C::CW, NP = CW / PC;
    const int q = warp & 3, group = (warp - 4) >> 2;
    uint8_t* const buf = sEpi + (warp - 4) * C::BUF;
    float* const sbias =
        reinterpret_cast<float*>(sEpi + C::EPI_WARPS * C::BUF + (warp - 4) * 128);
    const uint32_t tempty_pair = PAIR ? gb::mapa_shared(gb::smem_u32(tempty), 0) : 0u;
    int acc = 0;
    uint32_t acc_phase = 0;
    // what a tile reads is on its way before the tile's turn: its first block of the
    // residual and its biases (of the lane's column in each 32)
    uint32_t pre[16] = {};
    float bias[CW / 32];
    const auto row_of = [&](int u) {
      return ((u / p.n_tiles) * (PAIR ? 2 : 1) + (int)rank) * BM + q * 32;
    };
    const auto fetch_res = [&](int m0, int n0) {
      if (FLOAT && p.res && m0 < p.M && n0 < p.N)
        Block<T>::fetch(pre, static_cast<const T*>(p.res) + (long long)m0 * p.ldr + n0, p.ldr,
                        p.M - m0, p.N - n0, p.vec_r);
    };
    const auto fetch_bias = [&](int nb) {
#pragma unroll
      for (int i = 0; i < CW / 32; ++i) {
        const int n = nb + 32 * i + lane;
        bias[i] = p.bias && n < p.N ? p.bias[n] : 0.0f;
      }
    };
    const bool mine = !SPLIT || (warp - 4) % p.split == part;  // the block of the tile
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int m0 = row_of(unit0), nb = unit0 % p.n_tiles * BN + group * CW;
    if (mine && unit0 < units) {
      fetch_res(m0, nb);
      fetch_bias(nb);
    }
    for (int u = unit0; u < units; u += ustep) {
      const int un = u + ustep, m_next = un < units ? row_of(un) : p.M;
      const int nb_next = un % p.n_tiles * BN + group * CW;
      // SPLIT: a wait that ran out is in the error word, and the barriers are still met
      if (!gb::mbar_wait_bounded(&tfull[acc], acc_phase, p.wait_ns, p.err) && !SPLIT) break;
      gb::tc_fence_after();
      const uint32_t t = tmem + ((uint32_t)(q * 32) << 16) + acc * BN + group * CW;
      uint32_t r[CW / 32][32];
#pragma unroll
      for (int i = 0; i < CW / 32; ++i) gb::tmem_ld_x32(t + 32 * i, r[i]);
      gb::tmem_ld_wait();
      gb::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR)
          gb::mbar_arrive_cluster_control(tempty_pair + acc * 8);
        else
          gb::mbar_arrive(&tempty[acc]);
      }
      if constexpr (SPLIT) {
        static_assert(CW == 32, "a block");
        const int block = warp - 4, slots = (C::EPI_WARPS + p.split - 1) / p.split;
        const int owner = block % p.split, slot = block / p.split;
        // [range][slot][column][row]: a warp's store is 128 bytes in one piece (as 16-byte
        // pieces of rows 65 x 8192 x 2048 took 9.0 us, so 8.2 then, 7.6 now)
        float* const sums = reinterpret_cast<float*>(smem);
        static_assert(C::STAGES * C::STAGE_BYTES >= (16 + SPLIT_MOST - 1) * 4096, "sums");
        __syncwarp();
        gb::cluster_sync();  // every CTA's operands are read, and every CTA runs
        const uint32_t to = gb::mapa_shared(
            gb::smem_u32(sums + (part * slots + slot) * 1024 + lane), (uint32_t)owner);
#pragma unroll
        for (int i = 0; i < 32; ++i) gb::store_cluster(to + 128 * i, r[0][i]);
        gb::cluster_sync();
        if (mine) {
#pragma unroll
          for (int i = 0; i < 32; ++i) r[0][i] = 0u;
          for (int k = 0; k < p.split; ++k) {
            const float* const from = sums + (k * slots + slot) * 1024 + lane;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              r[0][i] = __float_as_uint(__uint_as_float(r[0][i]) + from[32 * i]);
          }
        }
      }
      if (mine && m0 < p.M) {
        uint32_t code[CW / 8], bytes = 0;  // of 4-bit outputs
#pragma unroll
        for (int s = 0; s < NP; ++s) {
          const int n0 = nb + PC * s;
          if (n0 >= p.N) {
            if (FLOAT) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) code[4 * s + i] = 0;
            continue;
          }
          if (PC * s % 32 == 0) {
            sbias[lane] = bias[PC * s / 32];
            __syncwarp();
          }
          const bool last = s + 1 == NP || n0 + PC >= p.N;  // of the tile's blocks
          if (last && un < units) fetch_bias(nb_next);
          float v[PC];
          const uint64_t al = pack2(p.alpha, p.alpha);
#pragma unroll
          for (int i = 0; i < PC; i += 4) {
            const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(sbias + PC * s % 32 + i);
            const uint32_t* const a = &r[PC * s / 32][PC * s % 32 + i];
            unpack2(fma2(pack2(__uint_as_float(a[0]), __uint_as_float(a[1])), al, b.x), v[i],
                    v[i + 1]);
            unpack2(fma2(pack2(__uint_as_float(a[2]), __uint_as_float(a[3])), al, b.y), v[i + 2],
                    v[i + 3]);
          }
          if constexpr (FLOAT) {
            finish_float<T>(p, &tm_y, v, buf, m0, n0, pre, [&] {
              if (last)
                fetch_res(m_next, nb_next);
              else
                fetch_res(m0, n0 + PC);
            });
          } else {
            activate<false>(v, p.act);
            uint32_t c[4], b;
            quantize32<FMT>(p.y_scale, v, p.N - n0, c, b);
#pragma unroll
            for (int i = 0; i < 4; ++i) code[4 * s + i] = c[i];
            bytes |= b << (s * (32 / kBlock<FMT>) * 8);
          }
          __syncwarp();
        }
        if (!FLOAT && m0 + lane < p.M && nb < p.N)
          store_codes<FMT, CW>(p, m0 + lane, nb, code, bytes);
      }
      if (m0 >= p.M || nb >= p.N) {  // nothing was read for this tile
        fetch_res(m_next, nb_next);
        if (un < units) fetch_bias(nb_next);
      }
      m0 = m_next;
      nb = nb_next;
      if (++acc == C::NACC) {
        acc = 0;
        acc_phase ^= 1;
      }
    }
    if (FLOAT && lane == 0) gb::bulk_wait_all();  // stores done before exit
  }
  gb::tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) gb::cluster_sync();
  if (warp == 0) {
    gb::tc_fence_after();
    if constexpr (PAIR)
      gb::tmem_dealloc_pair(tmem, 512);
    else
      gb::tmem_dealloc(tmem, 512);
  }
}

template <int FMT, int BN, bool PAIR, int YIO, bool SPLIT>
cudaError_t launch_tile(const Fp4Gemm& g, int split, cudaStream_t st) {
  using C = Cfg<FMT, BN, PAIR, YIO>;
  CUtensorMap tx, txs, tw, tws;
  if (!codes_map(&tx, g.x, g.M, g.C, BM) || !codes_map(&tw, g.w, g.K, g.C, C::BROWS) ||
      !scales_map(&txs, g.xs, FMT, g.M, g.C, C::ATOMS, 1) ||
      !scales_map(&tws, g.ws, FMT, g.K, g.C, C::ATOMS, C::PB))
    return cudaErrorInvalidValue;
  GemmParams p{};
  p.M = g.M;
  p.N = g.K;
  p.ksteps = gb_ceil_div(g.C, 256);
  p.kmmas_last = gb_ceil_div(g.C - (p.ksteps - 1) * 256, 64);
  p.m_tiles = (int)gb_ceil_div_ll(g.M, PAIR ? 2 * BM : BM);
  p.n_tiles = gb_ceil_div(g.K, BN);
  p.split = split;
  p.act = g.act;
  p.alpha = g.alpha;
  p.y_scale = tensor_scale(g.y_scale);
  p.bias = g.bias;
  p.res = g.res;
  p.y = g.y;
  p.ys = g.ys;
  p.ldr = g.ldr;
  p.ldy = g.ldy;
  if (YIO == CONV_FP4_IO_CODES) {
    p.vec_y = rows_vec<uint8_t>(g.y, code_pitch(g.K), 32);
  } else if (YIO == CONV_FP4_IO_BF16) {
    p.vec_y = rows_vec<__nv_bfloat16>(g.y, g.ldy, 16);
    p.vec_r = rows_vec<__nv_bfloat16>(g.res, g.ldr, 16);
  } else {
    p.vec_y = rows_vec<float>(g.y, g.ldy, 16);
    p.vec_r = rows_vec<float>(g.res, g.ldr, 16);
  }
  CUtensorMap ty = tx, tx64 = tx, tw64 = tw;
  if ((short_tail(g.M) && !codes_map(&tx64, g.x, g.M, g.C, 64)) ||
      (short_tail(g.K) && !codes_map(&tw64, g.w, g.K, g.C, 64)))
    return cudaErrorInvalidValue;
  if (YIO != CONV_FP4_IO_CODES && p.vec_y) {  // boxes of 32 rows x 64 bytes
    constexpr cuuint64_t es = YIO == CONV_FP4_IO_BF16 ? 2 : 4;
    cuuint64_t dims[2] = {(cuuint64_t)g.K, (cuuint64_t)g.M};
    cuuint64_t strides[1] = {(cuuint64_t)g.ldy * es};
    cuuint32_t box[2] = {(cuuint32_t)(64 / es), 32};
    cuuint32_t estr[2] = {1, 1};
    const CUtensorMapDataType dt =
        es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    if (gb_encode_tiled(&ty, dt, 2, g.y, dims, strides, box, estr, CU_TENSOR_MAP_SWIZZLE_64B) !=
        CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  p.err = gb_device_error_word();
  p.wait_ns = gb_wait_limit_ns();
  auto* kern = fp4_gemm_kernel<FMT, BN, PAIR, YIO, SPLIT>;
  cudaError_t e = gb_set_smem_once(reinterpret_cast<const void*>(kern), C::SMEM);
  if (e != cudaSuccess) return e;
  // the kernel's register split waits forever if it was launched with fewer
  static const int regs = [&] {
    cudaFuncAttributes fa = {};
    return cudaFuncGetAttributes(&fa, kern) == cudaSuccess ? fa.numRegs : 0;
  }();
  if (BN == 256 && regs * C::THREADS < 128 * 40 + 512 * 104) return cudaErrorLaunchOutOfResources;
  const long long units = (long long)p.m_tiles * p.n_tiles;
  if (units >= (1LL << 31)) return cudaErrorInvalidValue;
  const int cluster = PAIR ? 2 : split;  // split 1: no cluster
  const int grid =
      (int)std::min<long long>(units, SPLIT ? units : gb_num_sms() / cluster) * cluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kern, tx, txs, tw, tws, ty, tx64, tw64, p);
  if (e == cudaSuccess) gb_count_launch();
  return e;
}

// CTAs that share a tile: as many as all tiles' clusters find room for at once (more, and
// they run one after another: 65 x 8192 x 2048 by 8 14.6 us, by 4 7.6), if they save 14
// k-steps (0.2 us each); the exchange costs 2.5 us.
template <int FMT, int YIO>
int split_of(const Fp4Gemm& g, long long tiles) {
  using C = Cfg<FMT, 128, false, YIO>;
  auto* kern = fp4_gemm_kernel<FMT, 128, false, YIO, true>;
  const int ksteps = gb_ceil_div(g.C, 256);
  for (int s = SPLIT_MOST; s > 1; --s) {
    if (tiles * s > gb_num_sms() || ksteps - gb_ceil_div(ksteps, s) < 14) continue;
    if (tiles <= gb_active_clusters(reinterpret_cast<const void*>(kern), C::THREADS, C::SMEM, s))
      return s;
  }
  return 1;
}

template <int FMT, int YIO>
cudaError_t launch_y(const Fp4Gemm& g, cudaStream_t st) {
  // 128 x 128 tiles where they take one wave (256 x 2048 x 1000: 5.5 us against 7.7), or two
  // of up to 4 k-steps (2048 x 1024 x 2048 5.5 against 6.3); the SM pairs' tiles read half
  // the operands per product (8192 x 1024 x 4096 18.1 us against 21.3, 8192 x 4096 x 4096
  // 44.0 against 64.2)
  const long long tiles = gb_ceil_div_ll(g.M, 128) * gb_ceil_div_ll(g.K, 128);
  const int sms = gb_num_sms();
  const bool small = tiles <= sms || (tiles <= 2 * sms && g.C <= 1024) || g.K <= 128;
  if (!small) return launch_tile<FMT, 256, true, YIO, false>(g, 1, st);
  const int split = split_of<FMT, YIO>(g, tiles);
  return split > 1 ? launch_tile<FMT, 128, false, YIO, true>(g, split, st)
                   : launch_tile<FMT, 128, false, YIO, false>(g, 1, st);
}

template <int FMT>
cudaError_t launch_fmt(const Fp4Gemm& g, cudaStream_t st) {
  if (g.y_io == CONV_FP4_IO_BF16) return launch_y<FMT, CONV_FP4_IO_BF16>(g, st);
  if (g.y_io == CONV_FP4_IO_F32) return launch_y<FMT, CONV_FP4_IO_F32>(g, st);
  return launch_y<FMT, CONV_FP4_IO_CODES>(g, st);
}

}  // namespace

cudaError_t launch_fp4_gemm(const Fp4Gemm& g, cudaStream_t st) {
  return g.fmt == CONV_FP4_MX ? launch_fmt<CONV_FP4_MX>(g, st) : launch_fmt<CONV_FP4_NV>(g, st);
}
