"""Microscaled 4-bit matrices and the fully connected layer over them, as torch tensors.

Every computation is a call into libgbconv.so through ``binding`` (the formats and
their layout in memory: include/gbconv.h); memory and streams come from PyTorch.
"""
from __future__ import annotations

import contextlib
import threading

import torch

from . import binding as B


class Types(dict):
    def __missing__(self, t):
        raise ValueError(f"{t}: expected {', '.join(map(str, self))}")


CONV_DTYPE = Types({torch.bfloat16: B.CONV_BF16, torch.float32: B.CONV_F32})
IO = Types({torch.bfloat16: B.CONV_FP4_IO_BF16, torch.float32: B.CONV_FP4_IO_F32,
            None: B.CONV_FP4_IO_CODES})
BLOCK = {B.CONV_FP4_MX: 32, B.CONV_FP4_NV: 16}


# Handle of a device's current stream, without building a torch.cuda.Stream: a call's host
# time is a few microseconds in all, so its path here is kept short.
current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
current_device = getattr(torch._C, "_cuda_getDevice", None)


def call_stream(index, stream):
    """Stream handle (stream, or the current one for None) of a call on tensors of device
    index, which has to be the current GPU: the library launches there."""
    if index < 0:
        raise ValueError("tensors must be on the GPU")
    if index != current_device():
        raise ValueError(f"tensors on GPU {index}, but GPU {current_device()} is current")
    return current_stream(index) if stream is None else stream


def allocating_on(stream):
    """Context in which torch allocates for the stream handle (None: the current stream),
    so that memory freed by another stream's work is not handed out too early."""
    if stream is None or stream == torch.cuda.current_stream().cuda_stream:
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream))


class Workspaces:
    """Scratch memory of a layer's calls: a buffer per device and stream, whose calls follow
    each other.  A call that is captured into a CUDA graph gets memory of its own, from the
    graph's pool: the graph keeps the address, so it can be neither a buffer that a larger call
    replaces nor one that calls outside the graph write into."""

    __slots__ = ("_held",)

    def __init__(self):
        self._held = {}

    def get(self, need, device, index, stream, handle) -> torch.Tensor:
        if stream is None:
            return self._get(need, device, (index, handle))
        with allocating_on(stream):
            return self._get(need, device, (index, handle))

    def _get(self, need, device, key):
        if torch.cuda.is_current_stream_capturing():
            return torch.empty(need, dtype=torch.uint8, device=device)
        ws = self._held.get(key)
        if ws is None or ws.numel() < need:
            ws = self._held[key] = torch.empty(need, dtype=torch.uint8, device=device)
        return ws


def rows_of(t: torch.Tensor, cols: int, what: str):
    """(rows, elements between rows) of a tensor [..., cols] whose rows are evenly spaced."""
    shape = t.shape
    if shape[-1] != cols:
        raise ValueError(f"{what}: last dimension {shape[-1]}, expected {cols}")
    if t.is_contiguous():
        return t.numel() // cols, cols
    if t.dim() == 2:
        rows, ld = t.shape[0], t.stride(0)
        if t.stride(1) != 1 and cols > 1 and rows:
            raise ValueError(f"{what}: the elements of a row must be contiguous")
        if rows > 1 and ld < cols:
            raise ValueError(f"{what}: its rows overlap (an expanded tensor?)")
        return rows, ld if rows > 1 else cols
    raise ValueError(f"{what}: must be contiguous (or 2-D with contiguous rows)")


class Fp4Tensor:
    """A 4-bit matrix [rows][cols]: codes, scales (tiled, as conv_fp4_size says; contiguous
    uint8, of its bytes or more), tensor scale.  The tensors stay the ones it was made with
    (their addresses are kept)."""

    __slots__ = ("rows", "cols", "fmt", "tensor_scale", "codes", "scales", "shape", "codes_ptr",
                 "scales_ptr", "device", "index")

    def __init__(self, rows, cols, fmt, tensor_scale, codes, scales):
        if scales.get_device() != codes.get_device():
            raise ValueError("codes and scales: on different devices")
        if (codes.dtype is not torch.uint8 or scales.dtype is not torch.uint8
                or not codes.is_contiguous() or not scales.is_contiguous()
                or codes.numel() < rows * 16 * -(-cols // 32)
                or scales.numel() < -(-rows // 128) * -(-cols // (4 * BLOCK[fmt])) * 512):
            raise ValueError("codes, scales: expected contiguous uint8 of conv_fp4_size's bytes")
        self.rows, self.cols, self.fmt, self.tensor_scale = rows, cols, fmt, tensor_scale
        self.codes, self.scales = codes, scales
        self.shape = (rows, cols, fmt)
        self.codes_ptr, self.scales_ptr = codes.data_ptr(), scales.data_ptr()
        self.device, self.index = codes.device, codes.get_device()


def empty(rows, cols, fmt, device, tensor_scale=1.0, stream=None) -> Fp4Tensor:
    """An uninitialised 4-bit matrix."""
    cb, sb = B.conv_fp4_size(fmt, rows, cols)
    with allocating_on(stream):
        return Fp4Tensor(rows, cols, fmt, tensor_scale,
                         torch.empty(cb, dtype=torch.uint8, device=device),
                         torch.empty(sb, dtype=torch.uint8, device=device))


def quantize(x: torch.Tensor, fmt, tensor_scale=1.0, out: Fp4Tensor | None = None,
             stream=None) -> Fp4Tensor:
    """x [..., cols] (bf16 or fp32) in 4 bits."""
    cols = x.shape[-1]
    if x.is_contiguous() and cols:
        rows, ld = x.numel() // cols, cols
    else:
        rows, ld = rows_of(x, cols, "x")
    if out is None:
        out = empty(rows, cols, fmt, x.device, tensor_scale, stream)
    elif out.shape != (rows, cols, fmt):
        raise ValueError("out: a 4-bit matrix of another shape or format")
    index = out.index
    if x.get_device() != index:
        raise ValueError("x: on another device than out")
    B.conv_fp4_quantize(fmt, CONV_DTYPE[x.dtype], rows, cols, x.data_ptr(), ld, tensor_scale,
                        out.codes_ptr, out.scales_ptr, call_stream(index, stream))
    out.tensor_scale = tensor_scale
    return out


def dequantize(t: Fp4Tensor, dtype=torch.bfloat16, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """The values that t stands for, [rows][cols] in dtype (or out's)."""
    if out is None:
        with allocating_on(stream):
            out = torch.empty(t.rows, t.cols, dtype=dtype, device=t.device)
    rows, ld = rows_of(out, t.cols, "out")
    if rows != t.rows:
        raise ValueError(f"out: {rows} rows, expected {t.rows}")
    index = t.index
    if out.get_device() != index:
        raise ValueError("out: on another device than t")
    B.conv_fp4_dequantize(t.fmt, CONV_DTYPE[out.dtype], rows, t.cols, t.codes_ptr, t.scales_ptr,
                          t.tensor_scale, out.data_ptr(), ld, call_stream(index, stream))
    return out


class Fp4Linear:
    """y = act(x W^T + bias (+ residual)) with 4-bit x and W [K][C]; equally a 1x1
    convolution over NHWC pixels (x [..., C]).

    x_dtype: torch.bfloat16 or torch.float32 (quantised on the way in with tensor scale
    x_scale), or None for an ``Fp4Tensor``.  y_dtype: likewise, None gives an ``Fp4Tensor``
    with tensor scale y_scale.  Row strides of the tensors are followed.  Threads may share a
    layer."""

    def __init__(self, C, K, fmt=B.CONV_FP4_MX, x_dtype=torch.bfloat16, y_dtype=torch.bfloat16,
                 act=B.CONV_ACT_NONE, has_residual=False, x_scale=1.0, y_scale=1.0):
        self.C, self.K, self.fmt = C, K, fmt
        self.x_dtype, self.y_dtype = x_dtype, y_dtype
        self.x_scale, self.y_scale = x_scale, y_scale
        self.desc = B.conv_fp4_create(fmt, C, K, IO[x_dtype], IO[y_dtype])
        B.conv_fp4_set_epilogue(self.desc, act, has_residual)
        B.conv_fp4_set_tensor_scales(self.desc, x_scale, 1.0, y_scale)  # w's: with the weights
        self.w = None
        # a call gives the descriptor its strides and launches before another call, or other
        # weights, change them; calls on one stream share its workspace
        self._lock = threading.Lock()
        self._strides = (C, K, K)
        self._sizes = {}  # rows -> workspace bytes
        self._ws = Workspaces()

    def __del__(self):
        d = getattr(self, "desc", None)
        if d is not None:
            try:
                B.conv_fp4_destroy(d)
            except Exception:
                pass

    def prepack(self, w: torch.Tensor, w_scale=1.0, stream=None):
        """Quantise the weights [K][C] (bf16 or fp32) once."""
        if tuple(w.shape) != (self.K, self.C):
            raise ValueError(f"w: {tuple(w.shape)}, expected {(self.K, self.C)}")
        self._set(quantize(w, self.fmt, w_scale, stream=stream))

    def load(self, codes: torch.Tensor, scales: torch.Tensor, w_scale=1.0, stream=None):
        """Weights held in 4 bits: codes uint8 [K][16 * ceil(C / 32)], scales uint8
        [K][ceil(C / block)] row by row (a checkpoint's order; tiled here once)."""
        blocks = -(-self.C // BLOCK[self.fmt])
        if (tuple(codes.shape) != (self.K, 16 * -(-self.C // 32)) or codes.dtype != torch.uint8
                or not codes.is_contiguous()):
            raise ValueError("codes: expected contiguous uint8 [K][16 * ceil(C / 32)]")
        if (tuple(scales.shape) != (self.K, blocks) or scales.dtype != torch.uint8
                or not scales.is_contiguous()):
            raise ValueError("scales: expected contiguous uint8 [K][ceil(C / block)]")
        if scales.get_device() != codes.get_device():
            raise ValueError("codes and scales: on different devices")
        handle = call_stream(codes.get_device(), stream)
        _, sb = B.conv_fp4_size(self.fmt, self.K, self.C)
        with allocating_on(stream):
            tiled = torch.empty(sb, dtype=torch.uint8, device=codes.device)
        B.conv_fp4_pack_scales(self.fmt, self.K, self.C, scales.data_ptr(), tiled.data_ptr(),
                               handle)
        self._set(Fp4Tensor(self.K, self.C, self.fmt, w_scale, codes, tiled))

    def _set(self, w: Fp4Tensor):
        with self._lock:
            B.conv_fp4_set_tensor_scales(self.desc, self.x_scale, w.tensor_scale, self.y_scale)
            self.w = w

    def forward(self, x, bias=None, residual=None, out=None, stream=None):
        with self._lock:
            w = self.w
            if w is None:
                raise RuntimeError("prepack() or load() the weights first")
            C, K, y_dtype, index = self.C, self.K, self.y_dtype, w.index
            handle = call_stream(index, stream)
            bp = rp = xsp = ysp = None
            if self.x_dtype is None:
                if (x.cols, x.fmt, x.tensor_scale) != (C, self.fmt, self.x_scale):
                    raise ValueError("x: a 4-bit matrix of another width, format or tensor scale")
                if x.index != index:
                    raise ValueError("x: on another device than the weights")
                rows, ldx = x.rows, C
                xp, xsp = x.codes_ptr, x.scales_ptr
            else:
                if x.dtype is not self.x_dtype:
                    raise ValueError(f"x: {x.dtype}, expected {self.x_dtype}")
                if x.get_device() != index:
                    raise ValueError("x: on another device than the weights")
                rows, ldx = rows_of(x, C, "x")
                xp = x.data_ptr()
            if bias is not None:
                if bias.dtype is not torch.float32 or bias.numel() != K or not bias.is_contiguous():
                    raise ValueError("bias: expected contiguous fp32 [K]")
                if bias.get_device() != index:
                    raise ValueError("bias: on another device than the weights")
                bp = bias.data_ptr()
            ldr = ldy = K
            if y_dtype is None:
                if out is None:
                    out = empty(rows, K, self.fmt, w.device, self.y_scale, stream)
                elif out.shape != (rows, K, self.fmt):
                    raise ValueError("out: a 4-bit matrix of another shape or format")
                elif out.index != index:
                    raise ValueError("out: on another device than the weights")
                out.tensor_scale = self.y_scale
                yp, ysp = out.codes_ptr, out.scales_ptr
            else:
                if out is None:
                    lead = (rows,) if self.x_dtype is None else x.shape[:-1]
                    with allocating_on(stream):
                        out = torch.empty(*lead, K, dtype=y_dtype, device=w.device)
                elif out.get_device() != index:
                    raise ValueError("out: on another device than the weights")
                got, ldy = rows_of(out, K, "out")
                if got != rows or out.dtype is not y_dtype:
                    raise ValueError("out: another number of rows or type")
                yp = out.data_ptr()
            if residual is not None:
                got, ldr = rows_of(residual, K, "residual")
                if got != rows or residual.dtype is not y_dtype:
                    raise ValueError("residual: another number of rows or type than y")
                if residual.get_device() != index:
                    raise ValueError("residual: on another device than the weights")
                rp = residual.data_ptr()
            strides = (ldx, ldr, ldy)
            if strides != self._strides:
                B.conv_fp4_set_strides(self.desc, *strides)
                self._strides = strides
            need = self._sizes.get(rows)
            if need is None:
                need = self._sizes[rows] = B.conv_fp4_workspace_size(self.desc, rows)
            # held until the launches are enqueued
            ws = self._ws.get(need, w.device, index, stream, handle) if need else None
            B.conv_fp4_fwd(self.desc, rows, xp, xsp, w.codes_ptr, w.scales_ptr, bp, rp, yp, ysp,
                           ws.data_ptr() if need else None, need, handle)
            return out

    __call__ = forward
