// Product of two microscaled 4-bit matrices, y = act(alpha X W^T + bias + residual),
// on the block-scaled tcgen05 MMAs.
//
// GEMM names here: M rows of X, N rows of W (the layer's outputs), KR the reduction.
// Persistent CTAs of 192 threads: warp 0 loads (TMA), one thread of warp 1 copies the
// block scales to TMEM and issues the MMAs, warps 2..5 run the epilogue.  A k-step is
// 256 elements: 128-byte rows of codes (128-byte swizzle) and 512-byte scale tiles.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "fp4.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace {
using namespace gb::fp4;

constexpr int BM = 128;
constexpr int BKB = 128;  // bytes of a row per k-step: 256 codes

template <int FMT, int BN, bool PAIR>
struct Cfg {
  static constexpr int ATOMS = FMT == CONV_FP4_MX ? 2 : 4;  // scale tiles per panel and k-step
  static constexpr int PB = (BN + 127) / 128;               // 128-row panels of W
  static constexpr int BROWS = PAIR ? BN / 2 : BN;          // rows of W this CTA loads
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
  static constexpr int EPI_BYTES = 4 * 32 * 33 * 4;
  static constexpr int SMEM = STAGES * STAGE_BYTES + EPI_BYTES + 256 + 1024;
  static_assert(NACC * BN + STAGES * SF_COLS <= 512, "TMEM");
  static_assert(SMEM <= 232448, "shared memory");
};

struct GemmParams {
  int M, N, ksteps, kmmas_last;  // 64-element MMAs of the last k-step
  int m_tiles, n_tiles;          // PAIR: m_tiles counts 256-row units
  int act, y_io, fmt;
  float alpha, y_scale;
  const float* bias;
  const void* res;
  void* y;
  uint8_t* ys;
  long long ldr, ldy;
  int* err;
  unsigned long long wait_ns;
};

// Epilogue of a 32 x 32 block whose accumulators lie in the warp's staging buffer
// (row r, column c at stage[33 r + c]): a lane owns a column, rows go one by one, so
// that every access to the residual and the output is one segment per row.
template <typename T>
__device__ __forceinline__ void epilogue_float(const GemmParams& p, const float* stage, int m0,
                                               int n0) {
  const int lane = threadIdx.x & 31;
  const int n = n0 + lane;
  const bool live = n < p.N;
  const float b = p.bias && live ? p.bias[n] : 0.0f;
  const int rows = min(32, p.M - m0);
  const T* res = static_cast<const T*>(p.res);
  for (int r = 0; r < rows; ++r) {
    float v = stage[33 * r + lane] * p.alpha + b;
    if (!live) continue;
    if (res) v += load_f32(res + (long long)(m0 + r) * p.ldr + n);
    store_f32(static_cast<T*>(p.y) + (long long)(m0 + r) * p.ldy + n, activate(v, p.act));
  }
}

// The same block as 4-bit codes: a lane owns a row, whose 32 columns are one MX block
// or two NV blocks.
template <int FMT>
__device__ __forceinline__ void epilogue_codes(const GemmParams& p, const float* stage, int m0,
                                               int n0) {
  const int lane = threadIdx.x & 31;
  const long long m = m0 + lane;
  const long long pitch = code_pitch(p.N);
  const int tiles = tiles_per_row(FMT, p.N);
  if (m >= p.M || n0 >= p.N) return;
  float v[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const int n = n0 + i;
    const float b = p.bias && n < p.N ? p.bias[n] : 0.0f;
    v[i] = n < p.N ? activate(stage[33 * lane + i] * p.alpha + b, p.act) : 0.0f;
  }
  constexpr int B = kBlock<FMT>;
  uint32_t bytes = 0, code[4];
#pragma unroll
  for (int k = 0; k < 32 / B; ++k) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < B; ++i) top = max(top, abs_bits(v[k * B + i]));
    const BlockScale<FMT> s(__uint_as_float(top), p.y_scale);
    bytes |= s.byte << (8 * k);
#pragma unroll
    for (int i = 0; i < B / 8; ++i) {
      float e[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) e[t] = v[k * B + i * 8 + t];
      code[k * (B / 8) + i] = s.codes(e);
    }
  }
  *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.y) + m * pitch + n0 / 2) =
      make_uint4(code[0], code[1], code[2], code[3]);
  const int b0 = n0 / B;
  uint8_t* word = p.ys + scale_word_offset(m, b0 >> 2, tiles);
  if (FMT == CONV_FP4_MX)
    word[b0 & 3] = (uint8_t)bytes;
  else
    *reinterpret_cast<uint16_t*>(word + (b0 & 3)) = (uint16_t)bytes;
  // padding blocks of the row's last tile
  if (n0 + 32 >= p.N)
    for (int b = (n0 + 32) / B; (b >> 2) < tiles; ++b)
      p.ys[scale_word_offset(m, b >> 2, tiles) + (b & 3)] = 0;
}

template <int FMT, int BN, bool PAIR>
__global__ void __launch_bounds__(192, 1)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_xs,
                    const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_ws,
                    const GemmParams p) {
  using C = Cfg<FMT, BN, PAIR>;
  constexpr bool MX = FMT == CONV_FP4_MX;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + C::STAGES * C::A_BYTES;
  uint8_t* sFA = sB + C::STAGES * C::B_BYTES;
  uint8_t* sFB = sFA + C::STAGES * C::SFA_BYTES;
  float* sEpi = reinterpret_cast<float*>(sFB + C::STAGES * C::SFB_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(sEpi) + C::EPI_BYTES);
  uint64_t* empty = full + C::STAGES;
  uint64_t* tfull = empty + C::STAGES;
  uint64_t* tempty = tfull + C::NACC;
  uint64_t* mma_done = tempty + C::NACC;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? gb::cluster_ctarank() : 0u;
  const int unit0 = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
  const int ustep = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      gb::mbar_init(&full[s], 1);
      gb::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < C::NACC; ++b) {
      gb::mbar_init(&tfull[b], 1);
      gb::mbar_init(&tempty[b], PAIR ? 8 : 4);  // one arrival per epilogue warp
    }
    gb::mbar_init(mma_done, 1);
    gb::fence_barrier_init();
    gb::tma_prefetch_desc(&tm_x);
    gb::tma_prefetch_desc(&tm_w);
    gb::tma_prefetch_desc(&tm_xs);
    gb::tma_prefetch_desc(&tm_ws);
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
  const uint32_t tmem = *tmem_slot;
  gb::allow_dependents();

  const int units = p.m_tiles * p.n_tiles;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer ----------------
      int stage = 0;
      uint32_t phase = 0;
      long long issued = 0;
      bool ok = true;
      const uint32_t full_pair = PAIR ? gb::mapa_shared(gb::smem_u32(full), 0) : 0u;
      asm volatile("griddepcontrol.wait;" ::: "memory");
      for (int u = unit0; u < units && ok; u += ustep) {
        const int mt = (u / p.n_tiles) * (PAIR ? 2 : 1) + (int)rank, nt = u % p.n_tiles;
        const int brow = nt * BN + (PAIR ? (int)rank * C::BROWS : 0);
        for (int it = 0; it < p.ksteps; ++it) {
          if (!gb::mbar_wait_bounded(&empty[stage], phase ^ 1, p.wait_ns, p.err)) {
            ok = false;
            break;
          }
          uint8_t* const a = sA + stage * C::A_BYTES;
          uint8_t* const b = sB + stage * C::B_BYTES;
          uint8_t* const fa = sFA + stage * C::SFA_BYTES;
          uint8_t* const fb = sFB + stage * C::SFB_BYTES;
          const int sc = it * (C::ATOMS * 64);  // scale tiles as 8-byte elements
          if constexpr (PAIR) {
            if (rank == 0) gb::mbar_arrive_expect_tx(&full[stage], 2 * C::STAGE_BYTES);
            const uint32_t bar = full_pair + stage * 8;
            gb::tma_load_2d_pair(a, &tm_x, bar, it * BKB, mt * BM);
            gb::tma_load_2d_pair(b, &tm_w, bar, it * BKB, brow);
            gb::tma_load_2d_pair(fa, &tm_xs, bar, sc, mt);
            gb::tma_load_2d_pair(fb, &tm_ws, bar, sc, nt * BN / 128);
          } else {
            gb::mbar_arrive_expect_tx(&full[stage], C::STAGE_BYTES);
            gb::tma_load_2d(a, &tm_x, &full[stage], it * BKB, mt * BM);
            gb::tma_load_2d(b, &tm_w, &full[stage], it * BKB, brow);
            gb::tma_load_2d(fa, &tm_xs, &full[stage], sc, mt);
            gb::tma_load_2d(fb, &tm_ws, &full[stage], sc, nt * BN / 128);
          }
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
        gb::mbar_wait_bounded(&full[stage], phase, p.wait_ns, p.err);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // ---------------- scale copies and MMAs ----------------
      constexpr int MM = PAIR ? 2 * BM : BM;
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int u = unit0; u < units && ok; u += ustep) {
        if (!gb::mbar_wait_bounded(&tempty[acc], acc_phase ^ 1, p.wait_ns, p.err)) break;
        gb::tc_fence_after();
        const uint32_t d = tmem + acc * BN;
        for (int it = 0; it < p.ksteps; ++it) {
          const uint64_t ad = gb::sw128_kmajor_desc(gb::smem_u32(sA + stage * C::A_BYTES));
          const uint64_t bd = gb::sw128_kmajor_desc(gb::smem_u32(sB + stage * C::B_BYTES));
          const uint32_t fa = gb::smem_u32(sFA + stage * C::SFA_BYTES);
          const uint32_t fb = gb::smem_u32(sFB + stage * C::SFB_BYTES);
          const uint32_t sfa = tmem + C::NACC * BN + stage * C::SF_COLS;
          const uint32_t sfb = sfa + C::ATOMS * 4;
          if (!gb::mbar_wait_bounded(&full[stage], phase, p.wait_ns, p.err)) {
            ok = false;
            break;
          }
          gb::tc_fence_after();
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
          const int mmas = it + 1 < p.ksteps ? 4 : p.kmmas_last;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // MX: a scale word (4 blocks of 32) serves two MMAs; NV: (4 of 16) one
            const int j = MX ? k / 2 : k;
            const uint32_t id = gb::idesc_fp4(MM, BN, MX, MX ? (k & 1) * 2 : 0);
            if (k < mmas)
              gb::tc_mma_fp4<MX, PAIR>(d, ad + k * 2, bd + k * 2, id, sfa + 4 * j,
                                       sfb + 4 * j * C::PB, it > 0 || k > 0 ? 1u : 0u);
          }
          if constexpr (PAIR)
            gb::tc_commit_pair_multicast(&empty[stage], 0x3);
          else
            gb::tc_commit(&empty[stage]);
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if constexpr (PAIR)
          gb::tc_commit_pair_multicast(&tfull[acc], 0x3);
        else
          gb::tc_commit(&tfull[acc]);
        if (++acc == C::NACC) {
          acc = 0;
          acc_phase ^= 1;
        }
      }
      if constexpr (PAIR)
        gb::tc_commit_pair_multicast(mma_done, 0x1);
      else
        gb::tc_commit(mma_done);
      gb::mbar_wait_bounded(mma_done, 0, p.wait_ns, p.err);
    }
  } else {
    // ---------------- epilogue (warps 2..5) ----------------
    const int q = warp & 3;  // TMEM lane quarter this warp may access
    float* stage = sEpi + q * 32 * 33;
    const uint32_t tempty_pair = PAIR ? gb::mapa_shared(gb::smem_u32(tempty), 0) : 0u;
    int acc = 0;
    uint32_t acc_phase = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int u = unit0; u < units; u += ustep) {
      const int mt = (u / p.n_tiles) * (PAIR ? 2 : 1) + (int)rank, nt = u % p.n_tiles;
      const int m0 = mt * BM + q * 32, n0 = nt * BN;
      if (!gb::mbar_wait_bounded(&tfull[acc], acc_phase, p.wait_ns, p.err)) break;
      gb::tc_fence_after();
      const uint32_t t = tmem + ((uint32_t)(q * 32) << 16) + acc * BN;
#pragma unroll 1
      for (int c = 0; c < BN; c += 32) {
        uint32_t r[32];
        gb::tmem_ld_x32(t + c, r);
        gb::tmem_ld_wait();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 32; ++i) stage[33 * lane + i] = __uint_as_float(r[i]);
        __syncwarp();
        if (m0 < p.M && n0 + c < p.N) {
          if (p.y_io == CONV_FP4_IO_BF16)
            epilogue_float<__nv_bfloat16>(p, stage, m0, n0 + c);
          else if (p.y_io == CONV_FP4_IO_F32)
            epilogue_float<float>(p, stage, m0, n0 + c);
          else
            epilogue_codes<FMT>(p, stage, m0, n0 + c);
        }
      }
      gb::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR)
          gb::mbar_arrive_cluster(tempty_pair + acc * 8);
        else
          gb::mbar_arrive(&tempty[acc]);
      }
      if (++acc == C::NACC) {
        acc = 0;
        acc_phase ^= 1;
      }
    }
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

// [rows][pitch] bytes of codes in boxes of 128 bytes x box_rows
bool codes_map(CUtensorMap* map, const uint8_t* p, int rows, int cols, int box_rows) {
  cuuint64_t dims[2] = {(cuuint64_t)code_pitch(cols), (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)code_pitch(cols)};
  cuuint32_t box[2] = {BKB, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return gb_encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p), dims,
                         strides, box, estr, CU_TENSOR_MAP_SWIZZLE_128B) == CUDA_SUCCESS;
}
// scale tiles as [panels][tiles * 64] 8-byte elements, boxes of `atoms` tiles x `panels`
bool scales_map(CUtensorMap* map, const uint8_t* p, int fmt, int rows, int cols, int atoms,
                int box_panels) {
  const cuuint64_t w = (cuuint64_t)tiles_per_row(fmt, cols) * 64;
  cuuint64_t dims[2] = {w, (cuuint64_t)((rows + 127LL) / 128)};
  cuuint64_t strides[1] = {w * 8};
  cuuint32_t box[2] = {(cuuint32_t)(atoms * 64), (cuuint32_t)box_panels};
  cuuint32_t estr[2] = {1, 1};
  return gb_encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT64, 2, const_cast<uint8_t*>(p), dims,
                         strides, box, estr, CU_TENSOR_MAP_SWIZZLE_NONE) == CUDA_SUCCESS;
}

template <int FMT, int BN, bool PAIR>
cudaError_t launch_tile(const Fp4Gemm& g, cudaStream_t st) {
  using C = Cfg<FMT, BN, PAIR>;
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
  p.act = g.act;
  p.y_io = g.y_io;
  p.alpha = g.alpha;
  p.y_scale = g.y_scale;
  p.bias = g.bias;
  p.res = g.res;
  p.y = g.y;
  p.ys = g.ys;
  p.ldr = g.ldr;
  p.ldy = g.ldy;
  p.err = gb_device_error_word();
  p.wait_ns = gb_wait_limit_ns();
  auto* kern = fp4_gemm_kernel<FMT, BN, PAIR>;
  cudaError_t e = gb_set_smem_once(reinterpret_cast<const void*>(kern), C::SMEM);
  if (e != cudaSuccess) return e;
  const long long units = (long long)p.m_tiles * p.n_tiles;
  if (units >= (1LL << 31)) return cudaErrorInvalidValue;
  const int slots = PAIR ? gb_num_sms() / 2 : gb_num_sms();
  const int grid = (int)std::min<long long>(units, slots) * (PAIR ? 2 : 1);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(192);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = PAIR ? 2 : 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kern, tx, txs, tw, tws, p);
  if (e == cudaSuccess) gb_count_launch();
  return e;
}

template <int FMT>
cudaError_t launch_fmt(const Fp4Gemm& g, cudaStream_t st) {
  if (g.M > 128 && g.K > 128) return launch_tile<FMT, 256, true>(g, st);
  return launch_tile<FMT, 128, false>(g, st);
}

}  // namespace

cudaError_t launch_fp4_gemm(const Fp4Gemm& g, cudaStream_t st) {
  return g.fmt == CONV_FP4_MX ? launch_fmt<CONV_FP4_MX>(g, st) : launch_fmt<CONV_FP4_NV>(g, st);
}
