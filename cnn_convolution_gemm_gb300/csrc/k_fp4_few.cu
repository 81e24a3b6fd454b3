// Product of microscaled 4-bit matrices for few rows of X (one token to a small batch):
// y^T = W X^T, so that the tensor core's 128 rows are outputs and its N the few rows.
//
// Bound by the weights' bytes and by latency (one token through 4096 x 4096: 4.2 us with
// the weights in L2, 4.3 from HBM, whose bytes take 1.3; through 4096 -> 16384 8.4 from
// HBM, bytes 5.3; 32 rows through 8192 x 2048 5.5 us): a CTA streams 128 rows of W over a range of
// the reduction; the ranges of one tile are the CTAs of a cluster (up to 8), which
// add their partial sums through distributed shared memory in a fixed order.  Up to
// FUSED_ROWS rows of floating x are quantised on the way in, k-step by k-step, by
// the warps that later run the epilogue: one launch and no workspace.
//
// Warp 0 loads (TMA), warp 1 copies block scales and issues the MMAs (one elected lane),
// warps 4..7 quantise and run the epilogue.
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

constexpr int THREADS = 256;
constexpr int STAGES = 4;
constexpr int QUANT_WARPS = 4;  // that quantise a floating x, two rows each at a time
static_assert(FUSED_ROWS <= 2 * QUANT_WARPS, "rows past them would never be quantised");
constexpr int TMEM_COLS = 256;  // up to 128 of accumulator, 4 x 32 of scales

template <int FMT>
struct Cfg {
  static constexpr int ATOMS = FMT == CONV_FP4_MX ? 2 : 4;
  static constexpr int W_BYTES = 128 * BKB;
  static constexpr int SF_BYTES = ATOMS * 512;
  static constexpr int SF_COLS = ATOMS * 8;  // of W, then of X
  static constexpr int stage_bytes(int nt) { return W_BYTES + nt * BKB + 2 * SF_BYTES; }
  // ring, partial sums of the cluster, barriers, alignment
  static int smem(int nt, int split) {
    return STAGES * stage_bytes(nt) + (split > 1 ? 128 * 4 * nt : 0) + 256 + 1024;
  }
};

struct FewParams {
  int M, N, KR, nt;      // rows, outputs, reduction; rows rounded up to 8
  int ksteps, kmmas_last;
  int split_log2;        // CTAs of a cluster
  int warps_log2;        // FUSED: warps that quantise a k-step, up to QUANT_WARPS
  int act;
  float alpha;
  TensorScale x_scale, y_scale;
  const float* bias;
  const void *x, *res;   // x: floating x of the fused kernels
  int vec_x;
  void* y;
  uint8_t* ys;
  long long ldx, ldr, ldy;
  int* err;
  unsigned long long wait_ns;
};

// Output n of rows m, m + step, .. (rows of them); lanes of a warp are 32 consecutive
// outputs.
template <int FMT, int YIO>
__device__ __forceinline__ void finish(const FewParams& p, float (&v)[8], int m, int step, int rows,
                                       int n, float bias) {
  const bool live = n < p.N;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = fmaf(v[i], p.alpha, bias);
  if constexpr (YIO != CONV_FP4_IO_CODES) {
    using T = std::conditional_t<YIO == CONV_FP4_IO_BF16, __nv_bfloat16, float>;
    if (!live) return;
    if (p.res) {
      const T* const res = static_cast<const T*>(p.res) + m * p.ldr + n;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < rows) v[i] += load_f32(res + i * step * p.ldr);
    }
    activate<YIO == CONV_FP4_IO_F32>(v, p.act);
    T* const y = static_cast<T*>(p.y) + m * p.ldy + n;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < rows) store_f32(y + i * step * p.ldy, v[i]);
  } else {
    activate<false>(v, p.act);
    const int lane = threadIdx.x & 31;
    constexpr int B = kBlock<FMT>;
    const int n0 = n - lane, b = n / B, tiles = tiles_per_row(FMT, p.N);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= rows) break;
      const long long row = m + i * step;
      if (!live) v[i] = 0.0f;
      float top = fabsf(v[i]);
#pragma unroll
      for (int o = 1; o < B; o <<= 1) top = max_abs(top, top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
      const BlockScale<FMT> s(top, p.y_scale);
      // eight lanes' values in each of them
      float e[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) e[k] = __shfl_sync(0xFFFFFFFFu, v[i], (lane & 24) + k);
      const uint32_t code = s.codes(e);
      if ((lane & 7) == 0 && n0 < p.N)
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.y) + row * code_pitch(p.N) + n / 2) =
            code;
      if (lane % B == 0 && (b >> 2) < tiles)
        p.ys[scale_word_offset(row, b >> 2, tiles) + (b & 3)] = (uint8_t)s.byte;
    }
  }
}

// XIO: CONV_FP4_IO_CODES (tm_x, tm_xs) or the type of a floating x (M <= FUSED_ROWS).
template <int FMT, int XIO, int YIO>
__global__ void __launch_bounds__(THREADS)
    fp4_few_kernel(const __grid_constant__ CUtensorMap tm_w,
                   const __grid_constant__ CUtensorMap tm_ws,
                   const __grid_constant__ CUtensorMap tm_x,
                   const __grid_constant__ CUtensorMap tm_xs,
                   const __grid_constant__ CUtensorMap tm_w64, const FewParams p) {
  using C = Cfg<FMT>;
  constexpr bool MX = FMT == CONV_FP4_MX;
  constexpr bool FUSED = XIO != CONV_FP4_IO_CODES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int x_bytes = p.nt * BKB;
  const int split = 1 << p.split_log2;
  uint8_t* const sW = smem;
  uint8_t* const sX = sW + STAGES * C::W_BYTES;
  uint8_t* const sFW = sX + STAGES * x_bytes;
  uint8_t* const sFX = sFW + STAGES * C::SF_BYTES;
  float* const part = reinterpret_cast<float*>(sFX + STAGES * C::SF_BYTES);
  uint64_t* const full =
      reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(part) + (split > 1 ? 512 * p.nt : 0));
  uint64_t* const empty = full + STAGES;
  uint64_t* const tfull = empty + STAGES;
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(tfull + 1);

  const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0);  // uniform
  const int lane = threadIdx.x & 31;
  const int rank = blockIdx.x & (split - 1), tile = blockIdx.x >> p.split_log2;
  // this CTA's k-steps
  const int k0 = (int)((long long)p.ksteps * rank >> p.split_log2);
  const int k1 = (int)((long long)p.ksteps * (rank + 1) >> p.split_log2);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      // the loads, the quantising warps
      gb::mbar_init(&full[s], FUSED ? 1 + (1 << p.warps_log2) : 1);
      gb::mbar_init(&empty[s], 1);
    }
    gb::mbar_init(tfull, 1);
    gb::fence_barrier_init();
    gb::tma_prefetch_desc(&tm_w);
    gb::tma_prefetch_desc(&tm_ws);
    if (!FUSED) {
      gb::tma_prefetch_desc(&tm_x);
      gb::tma_prefetch_desc(&tm_xs);
    }
  }
  if (warp == 0) {
    gb::tmem_alloc(tmem_slot, TMEM_COLS);
    gb::tmem_relinquish();
  }
  gb::tc_fence_before();
  __syncthreads();
  if (split > 1) gb::cluster_sync();  // every CTA runs before another stores into it
  gb::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  gb::allow_dependents();

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    const bool one = gb::elect_one();
    int stage = 0;
    uint32_t phase = 0;
    int issued = 0;
    // the weights on their way to L2 while the kernel before this one ends (whatever it
    // still writes, L2 holds): 4096 x 4096 from HBM 4.9 -> 4.3 us a token
    for (int it = k0; it < k1 && it < k0 + STAGES; ++it)
      if (one) gb::tma_prefetch_2d(&tm_w, it * BKB, tile * 128);
    __syncwarp();
    const int wr = box_rows(tile * 128, p.N);
    const CUtensorMap* const wmap = wr == 64 ? &tm_w64 : &tm_w;
    const uint32_t tx = wr * BKB + C::SF_BYTES + (FUSED ? 0 : x_bytes + C::SF_BYTES);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int it = k0; it < k1; ++it) {
      if (!gb::mbar_wait_bounded_warp(&empty[stage], phase ^ 1, p.wait_ns, p.err)) break;
      if (one) {
        const int sc = it * (C::ATOMS * 64);  // scale tiles as 8-byte elements
        gb::mbar_arrive_expect_tx(&full[stage], tx);
        gb::tma_load_2d(sW + stage * C::W_BYTES, wmap, &full[stage], it * BKB, tile * 128);
        gb::tma_load_2d(sFW + stage * C::SF_BYTES, &tm_ws, &full[stage], sc, tile);
        if (!FUSED) {
          gb::tma_load_2d(sX + stage * x_bytes, &tm_x, &full[stage], it * BKB, 0);
          gb::tma_load_2d(sFX + stage * C::SF_BYTES, &tm_xs, &full[stage], sc, 0);
        }
      }
      __syncwarp();
      ++issued;
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1;
      }
    }
    // no copy into shared memory may be in flight at exit
    for (int i = issued < STAGES ? issued : STAGES; i > 0; --i) {
      if (--stage < 0) {
        stage = STAGES - 1;
        phase ^= 1;
      }
      gb::mbar_wait_bounded_warp(&full[stage], phase, p.wait_ns, p.err);
    }
  } else if (warp == 1) {
    // ---------------- scale copies and MMAs ----------------
    const bool one = gb::elect_one();
    int stage = 0;
    uint32_t phase = 0;
    for (int it = k0; it < k1; ++it) {
      if (!gb::mbar_wait_bounded_warp(&full[stage], phase, p.wait_ns, p.err)) break;
      gb::tc_fence_after();
      if (one) {
        const uint64_t wd = gb::sw128_kmajor_desc(gb::smem_u32(sW + stage * C::W_BYTES));
        const uint64_t xd = gb::sw128_kmajor_desc(gb::smem_u32(sX + stage * x_bytes));
        const uint32_t fw = gb::smem_u32(sFW + stage * C::SF_BYTES);
        const uint32_t fx = gb::smem_u32(sFX + stage * C::SF_BYTES);
        const uint32_t sfw = tmem + 128 + stage * C::SF_COLS, sfx = sfw + C::ATOMS * 4;
#pragma unroll
        for (int j = 0; j < C::ATOMS; ++j) {
          gb::tc_copy_scales<false>(sfw + 4 * j, gb::noswz_kmajor_desc(fw + j * 512, 128, 128));
          gb::tc_copy_scales<false>(sfx + 4 * j, gb::noswz_kmajor_desc(fx + j * 512, 128, 128));
        }
        const int mmas = it + 1 < p.ksteps ? 4 : p.kmmas_last;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int j = MX ? k / 2 : k;
          const uint32_t id = gb::idesc_fp4(128, p.nt, MX, MX ? (k & 1) * 2 : 0);
          if (k < mmas)
            gb::tc_mma_fp4<MX, false>(tmem, wd + k * 2, xd + k * 2, id, sfw + 4 * j, sfx + 4 * j,
                                      it > k0 || k > 0 ? 1u : 0u);
        }
        gb::tc_commit(&empty[stage]);
      }
      __syncwarp();
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (one) gb::tc_commit(tfull);
    __syncwarp();
    gb::mbar_wait_bounded_warp(tfull, 0, p.wait_ns, p.err);
  } else if (warp >= 4) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if constexpr (FUSED) {
      // ---------------- quantise x ----------------
      // 16 columns to a lane: a half-warp takes a row's 256 columns of a k-step, a warp two
      // rows; warps that are left over take other k-steps.  The next k-step's loads go out
      // before this one's arithmetic.
      using T = std::conditional_t<XIO == CONV_FP4_IO_BF16, __nv_bfloat16, float>;
      static_assert(QUANT_WARPS == 1 << 2 && QUANT_WARPS == THREADS / 32 - 4, "warps 4 and up");
      const int w = warp - 4, groups_log2 = 2 - p.warps_log2;
      const int r = (w & ((1 << p.warps_log2) - 1)) * 2 + (lane >> 4), gc = lane & 15;
      const T* const x = static_cast<const T*>(p.x) + (r < p.M ? r * p.ldx : 0);
      Raw16<T> next;
      int it = k0 + (w >> p.warps_log2);
      if (it < k1) next.load(x, it * 256 + gc * 16, p.KR, p.vec_x);
      for (; it < k1; it += 1 << groups_log2) {
        const Raw16<T> raw = next;
        const int stage = (it - k0) % STAGES;
        const uint32_t phase = ((it - k0) / STAGES) & 1;
        if (it + (1 << groups_log2) < k1)
          next.load(x, (it + (1 << groups_log2)) * 256 + gc * 16, p.KR, p.vec_x);
        if (!gb::mbar_wait_bounded_warp(&empty[stage], phase ^ 1, p.wait_ns, p.err)) break;
        float v[16];
        raw.get(v);
        uint2 code;
        uint32_t word;
        quantize16<FMT>(v, p.x_scale, code, word);
        if (r < p.M) {
          // row r of a 128-byte-swizzled tile; its scale words in tiles of 512 bytes
          *reinterpret_cast<uint2*>(sX + stage * x_bytes + r * BKB +
                                    (((gc >> 1) ^ (r & 7)) << 4) + (gc & 1) * 8) = code;
          constexpr int LT = 4 * kBlock<FMT> / 16;  // lanes of a scale tile
          if (gc % LT == 0)
            *reinterpret_cast<uint32_t*>(sFX + stage * C::SF_BYTES + gc / LT * 512 + r * 16) = word;
        }
        gb::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) gb::mbar_arrive(&full[stage]);
      }
    }
    // ---------------- accumulators: to the epilogue, or to the cluster ----------------
    gb::mbar_wait_bounded_warp(tfull, 0, p.wait_ns, p.err);
    gb::tc_fence_after();
    const uint32_t t = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const int o = (warp & 3) * 32 + lane, n = tile * 128 + o;
    if (split == 1) {
      const float bias = p.bias && n < p.N ? p.bias[n] : 0.0f;
      for (int c = 0; c < p.M; c += 8) {
        uint32_t r[8];
        gb::tmem_ld_x8(t + c, r);
        gb::tmem_ld_wait();
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
        finish<FMT, YIO>(p, v, c, 1, min(8, p.M - c), n, bias);
      }
    } else {
      // row m goes to CTA m % split, place m / split; source rank, place, output
      const int places = (p.M + split - 1) >> p.split_log2;
      const uint32_t mine = gb::smem_u32(part) + 4 * o + 512 * rank * places;
      for (int c = 0; c < p.M; c += 8) {
        uint32_t r[8];
        gb::tmem_ld_x8(t + c, r);
        gb::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int m = c + i;
          if (m < p.M)
            gb::store_cluster(gb::mapa_shared(mine + 512 * (m >> p.split_log2),
                                              (uint32_t)(m & (split - 1))),
                              r[i]);
        }
      }
    }
    gb::tc_fence_before();
  }
  __syncthreads();
  if (split > 1) {
    gb::cluster_sync();
    if (warp >= 4) {
      const int o = (warp & 3) * 32 + lane, n = tile * 128 + o;
      const float bias = p.bias && n < p.N ? p.bias[n] : 0.0f;
      const int places = (p.M + split - 1) >> p.split_log2;
      for (int i = 0; rank + i * split < p.M; i += 8) {
        float v[8] = {};
        const int rows = min(8, (p.M - rank - i * split + split - 1) >> p.split_log2);
        for (int r = 0; r < split; ++r) {
          const float* const from = part + 128 * (r * places + i) + o;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < rows) v[k] += from[128 * k];
        }
        finish<FMT, YIO>(p, v, rank + i * split, split, rows, n, bias);
      }
    }
  }
  if (warp == 0) {
    gb::tc_fence_after();
    gb::tmem_dealloc(tmem, TMEM_COLS);
  }
}

template <int FMT, int XIO, int YIO>
cudaError_t launch_t(const Fp4Gemm& g, cudaStream_t st) {
  using C = Cfg<FMT>;
  constexpr bool FUSED = XIO != CONV_FP4_IO_CODES;
  FewParams p{};
  p.M = g.M;
  p.N = g.K;
  p.KR = g.C;
  p.nt = gb_ceil_div(g.M, 8) * 8;
  p.ksteps = gb_ceil_div(g.C, 256);
  p.kmmas_last = gb_ceil_div(g.C - (p.ksteps - 1) * 256, 64);
  p.act = g.act;
  p.alpha = g.alpha;
  p.x_scale = tensor_scale(g.x_scale);
  p.y_scale = tensor_scale(g.y_scale);
  p.bias = g.bias;
  p.x = g.xf;
  p.res = g.res;
  p.y = g.y;
  p.ys = g.ys;
  p.ldx = g.ldx;
  p.ldr = g.ldr;
  p.ldy = g.ldy;
  p.vec_x = XIO == CONV_FP4_IO_BF16 ? rows_vec<__nv_bfloat16>(g.xf, g.ldx, 32)
                                    : rows_vec<float>(g.xf, g.ldx, 32);
  p.err = gb_device_error_word();
  p.wait_ns = gb_wait_limit_ns();
  // split the reduction while the tiles leave SMs idle and each CTA keeps two k-steps
  const int tiles = gb_ceil_div(g.K, 128);
  // (up to 8 CTAs; 4 where only one of them fits an SM: clusters of 8 then do not all find
  // room at once, 64 x 8192 x 2048 11.0 us against 5.3 with half the rows)
  const int most = 2 * (C::smem(p.nt, 8) + 1024) <= 228 * 1024 ? 3 : 2;
  p.split_log2 = 0;
  while (p.split_log2 < most && (tiles << (p.split_log2 + 1)) <= gb_num_sms() &&
         p.ksteps >> (p.split_log2 + 2))
    ++p.split_log2;
  const int split = 1 << p.split_log2;
  p.warps_log2 = 0;
  while ((1 << p.warps_log2) < QUANT_WARPS && (2 << p.warps_log2) < g.M) ++p.warps_log2;
  CUtensorMap tw, tws, tx, txs;
  if (!codes_map(&tw, g.w, g.K, g.C, 128) ||
      !scales_map(&tws, g.ws, FMT, g.K, g.C, C::ATOMS, 1))
    return cudaErrorInvalidValue;
  if (FUSED) {
    tx = tw;
    txs = tws;
  } else if (!codes_map(&tx, g.x, g.M, g.C, p.nt) ||
             !scales_map(&txs, g.xs, FMT, g.M, g.C, C::ATOMS, 1)) {
    return cudaErrorInvalidValue;
  }
  CUtensorMap tw64 = tw;
  if (short_tail(g.K) && !codes_map(&tw64, g.w, g.K, g.C, 64)) return cudaErrorInvalidValue;
  auto* kern = fp4_few_kernel<FMT, XIO, YIO>;
  const int smem = C::smem(p.nt, split);
  cudaError_t e = gb_set_smem_once(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * split));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kern, tw, tws, tx, txs, tw64, p);
  if (e == cudaSuccess) gb_count_launch();
  return e;
}

template <int FMT, int YIO>
cudaError_t launch_x(const Fp4Gemm& g, cudaStream_t st) {
  if (!g.xf) return launch_t<FMT, CONV_FP4_IO_CODES, YIO>(g, st);
  return g.x_io == CONV_FP4_IO_BF16 ? launch_t<FMT, CONV_FP4_IO_BF16, YIO>(g, st)
                                    : launch_t<FMT, CONV_FP4_IO_F32, YIO>(g, st);
}

template <int FMT>
cudaError_t launch_fmt(const Fp4Gemm& g, cudaStream_t st) {
  if (g.y_io == CONV_FP4_IO_BF16) return launch_x<FMT, CONV_FP4_IO_BF16>(g, st);
  if (g.y_io == CONV_FP4_IO_F32) return launch_x<FMT, CONV_FP4_IO_F32>(g, st);
  return launch_x<FMT, CONV_FP4_IO_CODES>(g, st);
}

}  // namespace

cudaError_t launch_fp4_few(const Fp4Gemm& g, cudaStream_t st) {
  return g.fmt == CONV_FP4_MX ? launch_fmt<CONV_FP4_MX>(g, st) : launch_fmt<CONV_FP4_NV>(g, st);
}
