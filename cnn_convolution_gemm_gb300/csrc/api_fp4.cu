// C-ABI entry points of the microscaled 4-bit matrices, their product and the norms
// around a residual block: argument checks, workspace layout, dispatch.
#include <cmath>
#include <cstring>
#include <new>

#include "fp4.cuh"
#include "internal.h"
#include "q8.cuh"

namespace {

constexpr int MOST = 1 << 30;  // rows and columns: tile arithmetic stays within an int

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t elem_bytes(int dtype) { return dtype == CONV_BF16 ? 2 : 4; }
bool is_float(int dtype) { return dtype == CONV_BF16 || dtype == CONV_F32; }
bool is_format(int fmt) { return fmt == CONV_FP4_MX || fmt == CONV_FP4_NV; }

conv_status_t cuda_status(cudaError_t e, const char* what) {
  return e == cudaSuccess ? gb_ok()
                          : gb_fail(CONV_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// CONV_OK or the failure for a tensor scale
conv_status_t check_scale(int fmt, float s, const char* what) {
  if (fmt == CONV_FP4_MX)
    return s == 1.0f ? CONV_OK
                     : gb_fail(CONV_ERR_BAD_PARAM, "%s must be 1 for CONV_FP4_MX", what);
  return s >= 1e-30f && s <= 1e30f
             ? CONV_OK
             : gb_fail(CONV_ERR_BAD_PARAM, "%s must lie in [1e-30, 1e30]", what);
}

size_t code_bytes(int rows, int cols) { return (size_t)rows * gb::fp4::code_pitch(cols); }
size_t scale_bytes(int fmt, int rows, int cols) {
  return ((size_t)rows + 127) / 128 * gb::fp4::tiles_per_row(fmt, cols) * 512;
}

// the checks that the matrix calls share
conv_status_t check_matrix(int fmt, int dtype, int rows, int cols, const void* t, long long* ld,
                           const char* tname, const void* codes, const void* scales) {
  if (!is_format(fmt)) return gb_fail(CONV_ERR_BAD_PARAM, "unknown 4-bit format %d", fmt);
  if (!is_float(dtype)) return gb_fail(CONV_ERR_BAD_PARAM, "%s must be bf16 or fp32", tname);
  if (rows < 0 || cols <= 0)
    return gb_fail(CONV_ERR_BAD_PARAM, "rows must be >= 0 and cols > 0");
  if (rows > MOST || cols > MOST)
    return gb_fail(CONV_ERR_UNSUPPORTED, "more than 2^30 rows or cols");
  if (*ld == 0) *ld = cols;
  if (*ld < cols) return gb_fail(CONV_ERR_BAD_PARAM, "row stride of %s below its row", tname);
  if (rows == 0) return CONV_OK;
  if (!t || !codes || !scales) return gb_fail(CONV_ERR_BAD_PARAM, "NULL tensor");
  if (!aligned(t, elem_bytes(dtype)))
    return gb_fail(CONV_ERR_ALIGNMENT, "%s must be aligned to its element", tname);
  if (!aligned(codes, 16) || !aligned(scales, 16))
    return gb_fail(CONV_ERR_ALIGNMENT, "codes and scales must be 16-byte aligned");
  return CONV_OK;
}

}  // namespace

extern "C" conv_status_t conv_fp4_size(conv_fp4_format_t fmt, int rows, int cols, size_t* cb,
                                       size_t* sb) {
  if (!cb || !sb) return gb_fail(CONV_ERR_BAD_PARAM, "NULL argument");
  if (!is_format(fmt)) return gb_fail(CONV_ERR_BAD_PARAM, "unknown 4-bit format %d", (int)fmt);
  if (rows < 0 || cols <= 0)
    return gb_fail(CONV_ERR_BAD_PARAM, "rows must be >= 0 and cols > 0");
  if (rows > MOST || cols > MOST)
    return gb_fail(CONV_ERR_UNSUPPORTED, "more than 2^30 rows or cols");
  *cb = code_bytes(rows, cols);
  *sb = scale_bytes(fmt, rows, cols);
  return gb_ok();
}

extern "C" conv_status_t conv_fp4_quantize(conv_fp4_format_t fmt, conv_dtype_t dtype, int rows,
                                           int cols, const void* x, long long ldx,
                                           float tensor_scale, void* codes, void* scales,
                                           void* stream) {
  conv_status_t st = check_matrix(fmt, dtype, rows, cols, x, &ldx, "x", codes, scales);
  if (st != CONV_OK) return st;
  if ((st = check_scale(fmt, tensor_scale, "tensor_scale")) != CONV_OK) return st;
  if (rows == 0) return gb_ok();
  return cuda_status(launch_fp4_quantize(fmt, dtype, rows, cols, x, ldx, tensor_scale, codes,
                                         scales, static_cast<cudaStream_t>(stream)),
                     "4-bit quantisation");
}

extern "C" conv_status_t conv_fp4_dequantize(conv_fp4_format_t fmt, conv_dtype_t dtype, int rows,
                                             int cols, const void* codes, const void* scales,
                                             float tensor_scale, void* y, long long ldy,
                                             void* stream) {
  conv_status_t st = check_matrix(fmt, dtype, rows, cols, y, &ldy, "y", codes, scales);
  if (st != CONV_OK) return st;
  if ((st = check_scale(fmt, tensor_scale, "tensor_scale")) != CONV_OK) return st;
  if (rows == 0) return gb_ok();
  return cuda_status(launch_fp4_dequantize(fmt, dtype, rows, cols, codes, scales, tensor_scale, y,
                                           ldy, static_cast<cudaStream_t>(stream)),
                     "4-bit dequantisation");
}

extern "C" conv_status_t conv_fp4_pack_scales(conv_fp4_format_t fmt, int rows, int cols,
                                              const void* src, void* scales, void* stream) {
  if (!is_format(fmt)) return gb_fail(CONV_ERR_BAD_PARAM, "unknown 4-bit format %d", (int)fmt);
  if (rows < 0 || cols <= 0)
    return gb_fail(CONV_ERR_BAD_PARAM, "rows must be >= 0 and cols > 0");
  if (rows > MOST || cols > MOST)
    return gb_fail(CONV_ERR_UNSUPPORTED, "more than 2^30 rows or cols");
  if (rows == 0) return gb_ok();
  if (!src || !scales) return gb_fail(CONV_ERR_BAD_PARAM, "NULL tensor");
  if (!aligned(scales, 16)) return gb_fail(CONV_ERR_ALIGNMENT, "scales must be 16-byte aligned");
  return cuda_status(launch_fp4_pack_scales(fmt, rows, cols, src, scales,
                                            static_cast<cudaStream_t>(stream)),
                     "scale packing");
}

// ---------------------------------------------------------------------------
// the product

extern "C" conv_status_t conv_fp4_create(conv_fp4_t* out, conv_fp4_format_t fmt, int C, int K,
                                         int x_io, int y_io) {
  if (!out) return gb_fail(CONV_ERR_BAD_PARAM, "out is NULL");
  *out = nullptr;
  if (!is_format(fmt)) return gb_fail(CONV_ERR_BAD_PARAM, "unknown 4-bit format %d", (int)fmt);
  if (C <= 0 || K <= 0) return gb_fail(CONV_ERR_BAD_PARAM, "sizes must be positive");
  if (C > MOST || K > MOST)
    return gb_fail(CONV_ERR_UNSUPPORTED, "more than 2^30 inputs or outputs");
  if (x_io < CONV_FP4_IO_BF16 || x_io > CONV_FP4_IO_CODES || y_io < CONV_FP4_IO_BF16 ||
      y_io > CONV_FP4_IO_CODES)
    return gb_fail(CONV_ERR_BAD_PARAM, "x_io and y_io must be 0, 1 or 2");
  gbconv_fp4_s* d = new (std::nothrow) gbconv_fp4_s{};
  if (!d) return gb_fail(CONV_ERR_BAD_PARAM, "out of host memory");
  d->fmt = fmt;
  d->C = C;
  d->K = K;
  d->x_io = x_io;
  d->y_io = y_io;
  d->x_scale = d->w_scale = d->y_scale = 1.0f;
  d->ldx = C;
  d->ldr = d->ldy = K;
  *out = d;
  return gb_ok();
}

extern "C" conv_status_t conv_fp4_destroy(conv_fp4_t d) {
  delete d;
  return gb_ok();
}

extern "C" conv_status_t conv_fp4_set_epilogue(conv_fp4_t d, int act, int has_residual) {
  if (!d) return gb_fail(CONV_ERR_BAD_PARAM, "desc is NULL");
  if (act < CONV_ACT_NONE || act > CONV_ACT_SILU)
    return gb_fail(CONV_ERR_BAD_PARAM, "act must be 0 .. 4");
  if (has_residual && d->y_io == CONV_FP4_IO_CODES)
    return gb_fail(CONV_ERR_UNSUPPORTED, "no residual with a 4-bit output");
  d->act = act;
  d->has_residual = has_residual ? 1 : 0;
  return gb_ok();
}

extern "C" conv_status_t conv_fp4_set_tensor_scales(conv_fp4_t d, float x, float w, float y) {
  if (!d) return gb_fail(CONV_ERR_BAD_PARAM, "desc is NULL");
  conv_status_t st;
  if ((st = check_scale(d->fmt, x, "the tensor scale of x")) != CONV_OK) return st;
  if ((st = check_scale(d->fmt, w, "the tensor scale of w")) != CONV_OK) return st;
  if ((st = check_scale(d->fmt, y, "the tensor scale of y")) != CONV_OK) return st;
  if (!(x * w >= 1e-37f && x * w <= 1e38f))
    return gb_fail(CONV_ERR_BAD_PARAM, "product of the tensor scales outside fp32");
  d->x_scale = x;
  d->w_scale = w;
  d->y_scale = y;
  return gb_ok();
}

extern "C" conv_status_t conv_fp4_set_strides(conv_fp4_t d, long long ldx, long long ldr,
                                              long long ldy) {
  if (!d) return gb_fail(CONV_ERR_BAD_PARAM, "desc is NULL");
  if (ldx && d->x_io == CONV_FP4_IO_CODES && ldx != d->C)
    return gb_fail(CONV_ERR_UNSUPPORTED, "4-bit x is contiguous");
  if (ldy && d->y_io == CONV_FP4_IO_CODES && ldy != d->K)
    return gb_fail(CONV_ERR_UNSUPPORTED, "4-bit y is contiguous");
  if ((ldx && ldx < d->C) || (ldr && ldr < d->K) || (ldy && ldy < d->K))
    return gb_fail(CONV_ERR_BAD_PARAM, "row stride below the row");
  d->ldx = ldx ? ldx : d->C;
  d->ldr = ldr ? ldr : d->K;
  d->ldy = ldy ? ldy : d->K;
  return gb_ok();
}

// workspace: codes of a float x, then its scales; none where the product quantises
static size_t fp4_workspace(const gbconv_fp4_s& d, int M) {
  if (d.x_io == CONV_FP4_IO_CODES || M <= FUSED_ROWS) return 0;
  return code_bytes(M, d.C) + scale_bytes(d.fmt, M, d.C);
}

extern "C" conv_status_t conv_fp4_workspace_size(conv_fp4_t d, int M, size_t* bytes) {
  if (!d || !bytes) return gb_fail(CONV_ERR_BAD_PARAM, "NULL argument");
  if (M < 0) return gb_fail(CONV_ERR_BAD_PARAM, "M must be >= 0");
  *bytes = fp4_workspace(*d, M);
  return gb_ok();
}

extern "C" conv_status_t conv_fp4_fwd(conv_fp4_t d, int M, const void* x, const void* x_scales,
                                      const void* w_codes, const void* w_scales, const float* bias,
                                      const void* residual, void* y, void* y_scales, void* ws,
                                      size_t ws_bytes, void* stream) {
  if (!d) return gb_fail(CONV_ERR_BAD_PARAM, "desc is NULL");
  if (M < 0) return gb_fail(CONV_ERR_BAD_PARAM, "M must be >= 0");
  if (M > MOST) return gb_fail(CONV_ERR_UNSUPPORTED, "more than 2^30 rows");
  if (M == 0) return gb_ok();
  const bool xc = d->x_io == CONV_FP4_IO_CODES, yc = d->y_io == CONV_FP4_IO_CODES;
  if (!x || !w_codes || !w_scales || !y) return gb_fail(CONV_ERR_BAD_PARAM, "NULL tensor");
  if (xc != (x_scales != nullptr) || yc != (y_scales != nullptr))
    return gb_fail(CONV_ERR_BAD_PARAM,
                   "x_scales / y_scales must be given exactly for a 4-bit x / y");
  if ((residual != nullptr) != (d->has_residual != 0))
    return gb_fail(CONV_ERR_BAD_PARAM,
                   "residual must be given exactly when the descriptor has one");
  const size_t xa = xc ? 16 : elem_bytes(d->x_io), ya = yc ? 16 : elem_bytes(d->y_io);
  if (!aligned(x, xa) || !aligned(y, ya) || !aligned(residual, ya) || !aligned(bias, 4))
    return gb_fail(CONV_ERR_ALIGNMENT, "a tensor is not aligned to its element (codes: 16 bytes)");
  if (!aligned(x_scales, 16) || !aligned(y_scales, 16) || !aligned(w_codes, 16) ||
      !aligned(w_scales, 16))
    return gb_fail(CONV_ERR_ALIGNMENT, "codes and scales must be 16-byte aligned");
  const size_t need = fp4_workspace(*d, M);
  if (need && (!ws || ws_bytes < need))
    return gb_fail(CONV_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                   ws ? ws_bytes : (size_t)0);
  if (!aligned(ws, 16)) return gb_fail(CONV_ERR_ALIGNMENT, "workspace must be 16-byte aligned");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Fp4Gemm g{};
  g.fmt = d->fmt;
  g.M = M;
  g.C = d->C;
  g.K = d->K;
  g.act = d->act;
  g.y_io = d->y_io;
  g.alpha = d->x_scale * d->w_scale;
  g.y_scale = d->y_scale;
  g.w = static_cast<const uint8_t*>(w_codes);
  g.ws = static_cast<const uint8_t*>(w_scales);
  g.bias = bias;
  g.res = residual;
  g.ldr = d->ldr;
  g.ldy = d->ldy;
  g.y = y;
  g.ys = static_cast<uint8_t*>(y_scales);
  g.x_scale = d->x_scale;
  if (!xc && M <= FUSED_ROWS) {
    g.xf = x;
    g.x_io = d->x_io;
    g.ldx = d->ldx;
  } else if (xc) {
    g.x = static_cast<const uint8_t*>(x);
    g.xs = static_cast<const uint8_t*>(x_scales);
  } else {
    uint8_t* codes = static_cast<uint8_t*>(ws);
    uint8_t* scales = codes + code_bytes(M, d->C);
    const cudaError_t e = launch_fp4_quantize(d->fmt, d->x_io, M, d->C, x, d->ldx, d->x_scale,
                                              codes, scales, st);
    if (e != cudaSuccess) return cuda_status(e, "4-bit quantisation");
    g.x = codes;
    g.xs = scales;
  }
  // Up to 32 rows on the kernel that splits the reduction; up to 64 where it is long and
  // the outputs few (64 x 8192 x 2048 6.9 us; 65 rows, on 128 x 128 tiles split over clusters, 7.6)
  static_assert(FUSED_ROWS <= 32, "only that kernel takes a floating x");
  const bool few =
      M <= 32 || (M <= 64 && d->C >= 4096 && 4LL * ((d->K + 127) / 128) <= gb_num_sms());
  return cuda_status(few ? launch_fp4_few(g, st) : launch_fp4_gemm(g, st), "4-bit product");
}

// ---------------------------------------------------------------------------
// norms around a residual block

struct gbconv_norm_s {
  NormArgs a;  // everything but rows and tensors; strides resolved
};

extern "C" conv_status_t conv_norm_create(conv_norm_t* out, int C, conv_dtype_t x_dtype,
                                          conv_dtype_t z_dtype) {
  if (!out) return gb_fail(CONV_ERR_BAD_PARAM, "out is NULL");
  *out = nullptr;
  if (C <= 0) return gb_fail(CONV_ERR_BAD_PARAM, "C must be positive");
  if (C > 32768) return gb_fail(CONV_ERR_UNSUPPORTED, "C above 32768");
  if (!is_float(x_dtype) || !is_float(z_dtype))
    return gb_fail(CONV_ERR_BAD_PARAM, "x_dtype and z_dtype must be bf16 or fp32");
  gbconv_norm_s* d = new (std::nothrow) gbconv_norm_s{};
  if (!d) return gb_fail(CONV_ERR_BAD_PARAM, "out of host memory");
  NormArgs& a = d->a;
  a.C = C;
  a.x_dtype = x_dtype;
  a.z_dtype = a.h_dtype = z_dtype;
  a.gate_rows = 1;
  a.rs = a.h_scale = 1.0f;
  a.ldx = a.ldz = a.ldg = a.ldxo = a.ldh = C;
  *out = d;
  return gb_ok();
}

extern "C" conv_status_t conv_norm_destroy(conv_norm_t d) {
  delete d;
  return gb_ok();
}

extern "C" conv_status_t conv_norm_set_z_dtype(conv_norm_t d, conv_dtype_t z_dtype) {
  if (!d) return gb_fail(CONV_ERR_BAD_PARAM, "desc is NULL");
  if (!is_float(z_dtype)) return gb_fail(CONV_ERR_BAD_PARAM, "z_dtype must be bf16 or fp32");
  if (z_dtype != d->a.h_dtype && (z_dtype != CONV_F32 || d->a.x_dtype != CONV_BF16))
    return gb_fail(CONV_ERR_UNSUPPORTED,
                   "z in another type than gate and h: fp32 with bf16 x, gate and h only");
  d->a.z_dtype = z_dtype;
  return gb_ok();
}

static conv_status_t check_norm(conv_norm_t d, int kind, float eps, const float* w,
                                const float* b) {
  if (!d) return gb_fail(CONV_ERR_BAD_PARAM, "desc is NULL");
  if (kind < CONV_NORM_NONE || kind > CONV_NORM_LAYER)
    return gb_fail(CONV_ERR_BAD_PARAM, "unknown norm %d", kind);
  if (!(eps >= 0.0f && eps < INFINITY)) return gb_fail(CONV_ERR_BAD_PARAM, "eps must be >= 0");
  if (kind == CONV_NORM_NONE && (w || b))
    return gb_fail(CONV_ERR_BAD_PARAM, "w and b belong to a norm");
  if (b && kind != CONV_NORM_LAYER)
    return gb_fail(CONV_ERR_UNSUPPORTED, "b belongs to a layer norm");
  if (!aligned(w, 4) || !aligned(b, 4))
    return gb_fail(CONV_ERR_ALIGNMENT, "w and b must be aligned to their elements");
  return CONV_OK;
}

extern "C" conv_status_t conv_norm_set_post(conv_norm_t d, int kind, float eps, const float* w,
                                            const float* b) {
  const conv_status_t st = check_norm(d, kind, eps, w, b);
  if (st != CONV_OK) return st;
  d->a.post = kind;
  d->a.eps_post = eps;
  d->a.w_post = w;
  d->a.b_post = b;
  return gb_ok();
}

extern "C" conv_status_t conv_norm_set_pre(conv_norm_t d, int kind, float eps, const float* w,
                                           const float* b) {
  const conv_status_t st = check_norm(d, kind, eps, w, b);
  if (st != CONV_OK) return st;
  d->a.pre = kind;
  d->a.eps_pre = eps;
  d->a.w_pre = w;
  d->a.b_pre = b;
  return gb_ok();
}

extern "C" conv_status_t conv_norm_set_gate(conv_norm_t d, int gate, int gate_rows,
                                            float residual_scale) {
  if (!d) return gb_fail(CONV_ERR_BAD_PARAM, "desc is NULL");
  if (gate < CONV_GATE_NONE || gate > CONV_GATE_SIGMOID)
    return gb_fail(CONV_ERR_BAD_PARAM, "unknown gate %d", gate);
  if (gate_rows <= 0) return gb_fail(CONV_ERR_BAD_PARAM, "gate_rows must be positive");
  if (!std::isfinite(residual_scale))
    return gb_fail(CONV_ERR_BAD_PARAM, "residual_scale must be finite");
  d->a.gate_kind = gate;
  d->a.gate_rows = gate_rows;
  d->a.rs = residual_scale;
  return gb_ok();
}

extern "C" conv_status_t conv_norm_set_output(conv_norm_t d, int out, float tensor_scale) {
  if (!d) return gb_fail(CONV_ERR_BAD_PARAM, "desc is NULL");
  if (out < CONV_NORM_OUT_FLOAT || out > CONV_NORM_OUT_FP4_NV)
    return gb_fail(CONV_ERR_BAD_PARAM, "unknown output %d", out);
  const conv_status_t st =
      check_scale(out == CONV_NORM_OUT_FP4_NV ? CONV_FP4_NV : CONV_FP4_MX, tensor_scale,
                  "tensor_scale");
  if (st != CONV_OK) return st;
  d->a.out = out;
  d->a.h_scale = tensor_scale;
  return gb_ok();
}

extern "C" conv_status_t conv_norm_set_output_q8(conv_norm_t d, conv_q8_format_t fmt, int group) {
  if (!d) return gb_fail(CONV_ERR_BAD_PARAM, "desc is NULL");
  if (fmt != CONV_Q8_E4M3 && fmt != CONV_Q8_INT8)
    return gb_fail(CONV_ERR_BAD_PARAM, "unknown 8-bit format %d", (int)fmt);
  if (group != 0 && group != gb::q8::GROUP)
    return gb_fail(CONV_ERR_BAD_PARAM, "group must be 0 or 128");
  d->a.out = fmt == CONV_Q8_E4M3 ? NORM_OUT_Q8_E4M3 : NORM_OUT_Q8_INT8;
  d->a.h_group = group;
  d->a.h_scale = 1.0f;
  return gb_ok();
}

extern "C" conv_status_t conv_norm_set_strides(conv_norm_t d, long long ldx, long long ldz,
                                               long long ldg, long long ldxo, long long ldh) {
  if (!d) return gb_fail(CONV_ERR_BAD_PARAM, "desc is NULL");
  const long long ld[5] = {ldx, ldz, ldg, ldxo, ldh};
  for (long long v : ld)
    if (v && v < d->a.C) return gb_fail(CONV_ERR_BAD_PARAM, "row stride below the row");
  long long* const to[5] = {&d->a.ldx, &d->a.ldz, &d->a.ldg, &d->a.ldxo, &d->a.ldh};
  for (int i = 0; i < 5; ++i) *to[i] = ld[i] ? ld[i] : d->a.C;
  return gb_ok();
}

// the arguments of a norm's launch, or why there is none
static conv_status_t check_norm_call(conv_norm_t d, int rows, const void* x, const void* z,
                                     const void* gate, void* x_out, void* h, void* h_scales,
                                     NormArgs* to) {
  NormArgs& a = *to;
  a = d->a;
  if (!x) return gb_fail(CONV_ERR_BAD_PARAM, "x is NULL");
  if (!x_out && !h) return gb_fail(CONV_ERR_BAD_PARAM, "no output");
  if ((h != nullptr) != (a.pre != CONV_NORM_NONE))
    return gb_fail(CONV_ERR_BAD_PARAM, "h must be given exactly when there is a norm before");
  const bool codes = a.out != CONV_NORM_OUT_FLOAT;
  if ((h_scales != nullptr) != (h != nullptr && codes))
    return gb_fail(CONV_ERR_BAD_PARAM, "h_scales must be given exactly for a 4- or 8-bit h");
  if ((gate != nullptr) != (z != nullptr && a.gate_kind != CONV_GATE_NONE))
    return gb_fail(CONV_ERR_BAD_PARAM,
                   "gate must be given exactly when the descriptor has one and z is given");
  if (codes && a.ldh != a.C) return gb_fail(CONV_ERR_UNSUPPORTED, "4- and 8-bit h are contiguous");
  const size_t xb = elem_bytes(a.x_dtype), hb = elem_bytes(a.h_dtype);
  if (!aligned(x, xb) || !aligned(x_out, xb) || !aligned(z, elem_bytes(a.z_dtype)) ||
      !aligned(gate, hb) || !aligned(h, codes ? 16 : hb) || !aligned(h_scales, 16))
    return gb_fail(CONV_ERR_ALIGNMENT, "a tensor is not aligned to its element (codes: 16 bytes)");
  if (x_out == x && a.ldxo != a.ldx)
    return gb_fail(CONV_ERR_BAD_PARAM, "x_out may be x only with x's row stride");
  a.rows = rows;
  a.x = x;
  a.z = z;
  a.gate = gate;
  a.x_out = x_out;
  a.h = h;
  a.hs = static_cast<uint8_t*>(h_scales);
  a.err = gb_device_error_word();
  a.wait_ns = gb_wait_limit_ns();
  return CONV_OK;
}

static conv_status_t launch_norm(const NormArgs& a, cudaStream_t st) {
  const bool q8 = a.out == NORM_OUT_Q8_E4M3 || a.out == NORM_OUT_Q8_INT8;
  // without z its type does not matter
  if (a.z && a.z_dtype != a.h_dtype)
    return cuda_status(q8 ? launch_norm_q8_bfb(a, st) : launch_norm_bfb(a, st), "norm");
  const bool xb16 = a.x_dtype == CONV_BF16, zb16 = a.h_dtype == CONV_BF16;
  if (q8)
    return cuda_status(xb16 ? (zb16 ? launch_norm_q8_bb(a, st) : launch_norm_q8_bf(a, st))
                            : (zb16 ? launch_norm_q8_fb(a, st) : launch_norm_q8_ff(a, st)),
                       "norm");
  return cuda_status(xb16 ? (zb16 ? launch_norm_bb(a, st) : launch_norm_bf(a, st))
                          : (zb16 ? launch_norm_fb(a, st) : launch_norm_ff(a, st)),
                     "norm");
}

extern "C" conv_status_t conv_norm_fwd(conv_norm_t d, int rows, const void* x, const void* z,
                                       const void* gate, void* x_out, void* h, void* h_scales,
                                       void* stream) {
  if (!d) return gb_fail(CONV_ERR_BAD_PARAM, "desc is NULL");
  if (rows < 0) return gb_fail(CONV_ERR_BAD_PARAM, "rows must be >= 0");
  if (rows == 0) return gb_ok();
  NormArgs a;
  const conv_status_t st = check_norm_call(d, rows, x, z, gate, x_out, h, h_scales, &a);
  return st != CONV_OK ? st : launch_norm(a, static_cast<cudaStream_t>(stream));
}

// ---------------------------------------------------------------------------
// a residual block

struct gbconv_fp4_block_s {
  conv_norm_t norm_in, norm_out;
  conv_fp4_t fc1, fc2;
  const void *w1, *s1, *w2, *s2;
  const float *b1, *b2;
};

namespace {

// parts of the workspace, each on a 256-byte boundary
struct BlockParts {
  size_t h, hs, t, ts, z, bytes;
};
BlockParts block_parts(const gbconv_fp4_block_s& b, int M) {
  BlockParts p;
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t from = at;
    at += (bytes + 255) / 256 * 256;
    return from;
  };
  p.h = take(code_bytes(M, b.fc1->C));
  p.hs = take(scale_bytes(b.fc1->fmt, M, b.fc1->C));
  p.t = take(code_bytes(M, b.fc1->K));
  p.ts = take(scale_bytes(b.fc1->fmt, M, b.fc1->K));
  p.z = take((size_t)M * b.fc2->K * elem_bytes(b.fc2->y_io));
  p.bytes = at;
  return p;
}

// whether the descriptors, as they are now, fit together
conv_status_t check_block(const gbconv_fp4_block_s& b) {
  const NormArgs &in = b.norm_in->a, &out = b.norm_out->a;
  const gbconv_fp4_s &f1 = *b.fc1, &f2 = *b.fc2;
  const char* wrong = nullptr;
  if (in.C != f1.C || f1.K != f2.C || f2.K != out.C || in.C != out.C)
    wrong = "widths do not fit";
  else if (f1.x_io != CONV_FP4_IO_CODES || f1.y_io != CONV_FP4_IO_CODES ||
           f2.x_io != CONV_FP4_IO_CODES || f2.y_io == CONV_FP4_IO_CODES)
    wrong = "the layers pass 4 bits on, the second gives floats";
  else if (f1.fmt != f2.fmt ||
           in.out != (f1.fmt == CONV_FP4_MX ? CONV_NORM_OUT_FP4_MX : CONV_NORM_OUT_FP4_NV))
    wrong = "formats do not fit";
  else if (in.h_scale != f1.x_scale || f1.y_scale != f2.x_scale)
    wrong = "tensor scales do not fit";
  else if (in.pre == CONV_NORM_NONE || in.x_dtype != out.x_dtype || in.ldx != out.ldx)
    wrong = "the norms do not read the same x";
  else if (f2.y_io != out.z_dtype || f2.ldy != out.C || out.ldz != out.C)
    wrong = "z is contiguous, in the second norm's z_dtype";
  else if (f1.has_residual || f2.has_residual)
    wrong = "a layer has a residual of its own";
  return wrong ? gb_fail(CONV_ERR_BAD_PARAM, "residual block: %s", wrong) : CONV_OK;
}

}  // namespace

static_assert((int)CONV_FP4_IO_BF16 == (int)CONV_BF16 && (int)CONV_FP4_IO_F32 == (int)CONV_F32,
              "check_block, elem_bytes");

extern "C" conv_status_t conv_fp4_block_create(conv_fp4_block_t* out, conv_norm_t norm_in,
                                               conv_fp4_t fc1, conv_fp4_t fc2,
                                               conv_norm_t norm_out) {
  if (!out) return gb_fail(CONV_ERR_BAD_PARAM, "out is NULL");
  *out = nullptr;
  if (!norm_in || !fc1 || !fc2 || !norm_out)
    return gb_fail(CONV_ERR_BAD_PARAM, "a descriptor is NULL");
  const gbconv_fp4_block_s b{norm_in, norm_out, fc1, fc2};
  const conv_status_t st = check_block(b);
  if (st != CONV_OK) return st;
  *out = new (std::nothrow) gbconv_fp4_block_s(b);
  return *out ? gb_ok() : gb_fail(CONV_ERR_BAD_PARAM, "out of host memory");
}

extern "C" conv_status_t conv_fp4_block_destroy(conv_fp4_block_t d) {
  delete d;
  return gb_ok();
}

extern "C" conv_status_t conv_fp4_block_set_weights(conv_fp4_block_t d, const void* w1,
                                                    const void* s1, const float* b1,
                                                    const void* w2, const void* s2,
                                                    const float* b2) {
  if (!d) return gb_fail(CONV_ERR_BAD_PARAM, "desc is NULL");
  if (!w1 || !s1 || !w2 || !s2) return gb_fail(CONV_ERR_BAD_PARAM, "NULL tensor");
  if (!aligned(w1, 16) || !aligned(s1, 16) || !aligned(w2, 16) || !aligned(s2, 16))
    return gb_fail(CONV_ERR_ALIGNMENT, "codes and scales must be 16-byte aligned");
  if (!aligned(b1, 4) || !aligned(b2, 4))
    return gb_fail(CONV_ERR_ALIGNMENT, "biases must be aligned to their elements");
  d->w1 = w1;
  d->s1 = s1;
  d->b1 = b1;
  d->w2 = w2;
  d->s2 = s2;
  d->b2 = b2;
  return gb_ok();
}

extern "C" conv_status_t conv_fp4_block_workspace_size(conv_fp4_block_t d, int M, size_t* bytes) {
  if (!d || !bytes) return gb_fail(CONV_ERR_BAD_PARAM, "NULL argument");
  if (M < 0) return gb_fail(CONV_ERR_BAD_PARAM, "M must be >= 0");
  if (M > MOST) return gb_fail(CONV_ERR_UNSUPPORTED, "more than 2^30 rows");
  *bytes = block_parts(*d, M).bytes;
  return gb_ok();
}

extern "C" conv_status_t conv_fp4_block_fwd(conv_fp4_block_t d, int M, const void* x,
                                            const void* h, const void* h_scales, const void* gate,
                                            void* x_out, void* h_out, void* h_out_scales, void* ws,
                                            size_t ws_bytes, void* stream) {
  if (!d) return gb_fail(CONV_ERR_BAD_PARAM, "desc is NULL");
  if (M < 0) return gb_fail(CONV_ERR_BAD_PARAM, "M must be >= 0");
  if (M > MOST) return gb_fail(CONV_ERR_UNSUPPORTED, "more than 2^30 rows");
  conv_status_t st = check_block(*d);
  if (st != CONV_OK) return st;
  if (M == 0) return gb_ok();
  if (!d->w1) return gb_fail(CONV_ERR_BAD_PARAM, "no weights yet");
  if ((h != nullptr) != (h_scales != nullptr))
    return gb_fail(CONV_ERR_BAD_PARAM, "h and h_scales come together");
  const BlockParts p = block_parts(*d, M);
  if (!ws || ws_bytes < p.bytes)
    return gb_fail(CONV_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", p.bytes,
                   ws ? ws_bytes : (size_t)0);
  if (!aligned(ws, 16)) return gb_fail(CONV_ERR_ALIGNMENT, "workspace must be 16-byte aligned");
  // the last call's checks first, so that a refusal enqueues nothing
  char* const w = static_cast<char*>(ws);
  NormArgs out;
  if ((st = check_norm_call(d->norm_out, M, x, w + p.z, gate, x_out, h_out, h_out_scales, &out)) !=
      CONV_OK)
    return st;
  if (!h) {
    if ((st = conv_norm_fwd(d->norm_in, M, x, nullptr, nullptr, nullptr, w + p.h, w + p.hs,
                            stream)) != CONV_OK)
      return st;
    h = w + p.h;
    h_scales = w + p.hs;
  }
  if ((st = conv_fp4_fwd(d->fc1, M, h, h_scales, d->w1, d->s1, d->b1, nullptr, w + p.t, w + p.ts,
                         nullptr, 0, stream)) != CONV_OK ||
      (st = conv_fp4_fwd(d->fc2, M, w + p.t, w + p.ts, d->w2, d->s2, d->b2, nullptr, w + p.z,
                         nullptr, nullptr, 0, stream)) != CONV_OK)
    return st;
  return launch_norm(out, static_cast<cudaStream_t>(stream));
}
