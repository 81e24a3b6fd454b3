"""The pass between two residual blocks as a torch-facing layer (conv_norm_* of gbconv.h)."""
from __future__ import annotations

import threading

import torch

from . import binding as B
from . import fp4
from .fp4 import CONV_DTYPE, allocating_on, call_stream, rows_of


class ResidualNorm:
    """u = norm_post(z);  x' = x + residual_scale * g(gate) * u;  h = norm_pre(x').

    post, pre: binding.CONV_NORM_*; w_*, b_*: fp32 [C] or None.  gate: binding.CONV_GATE_*,
    one row of gates for gate_rows consecutive rows.  dtype: of x and x'; z_dtype: of z (dtype
    if None); h_dtype: of gate and h (z_dtype if None, else bf16 with bf16 x and fp32 z).  h_fmt: binding.CONV_FP4_* gives h as an ``Fp4Tensor`` with
    tensor scale h_scale.  Row strides of 2-D tensors are followed.  Threads may share a
    layer."""

    def __init__(self, C, dtype=torch.bfloat16, z_dtype=None, eps=1e-6, post=B.CONV_NORM_NONE,
                 w_post=None, b_post=None, pre=B.CONV_NORM_NONE, w_pre=None, b_pre=None,
                 gate=B.CONV_GATE_NONE, gate_rows=1, residual_scale=1.0, h_fmt=None, h_scale=1.0,
                 h_dtype=None):
        self.C, self.dtype, self.z_dtype = C, dtype, dtype if z_dtype is None else z_dtype
        self.h_dtype = self.z_dtype if h_dtype is None else h_dtype
        self.post, self.pre, self.gate, self.gate_rows = post, pre, gate, gate_rows
        self.h_fmt, self.h_scale = h_fmt, h_scale
        self._params = (w_post, b_post, w_pre, b_pre)  # the descriptor holds their addresses
        self.index = None  # the device of the weights; None: there are none
        for p in self._params:
            if p is None:
                continue
            if p.dtype != torch.float32 or p.numel() != C or not p.is_contiguous():
                raise ValueError("weights and biases: expected contiguous fp32 [C]")
            if p.get_device() < 0 or self.index not in (None, p.get_device()):
                raise ValueError("weights and biases: must be on one GPU")
            self.index = p.get_device()
        wp, bp, wq, bq = (None if p is None else p.data_ptr() for p in self._params)
        self.desc = B.conv_norm_create(C, CONV_DTYPE[dtype], CONV_DTYPE[self.h_dtype])
        B.conv_norm_set_z_dtype(self.desc, CONV_DTYPE[self.z_dtype])
        B.conv_norm_set_post(self.desc, post, eps, wp, bp)
        B.conv_norm_set_pre(self.desc, pre, eps, wq, bq)
        B.conv_norm_set_gate(self.desc, gate, gate_rows, residual_scale)
        if h_fmt is not None:
            B.conv_norm_set_output(self.desc, B.CONV_NORM_OUT_FP4_MX if h_fmt == B.CONV_FP4_MX
                                   else B.CONV_NORM_OUT_FP4_NV, h_scale)
        # a call gives the descriptor its strides and launches before another call changes them
        self._lock = threading.Lock()
        self._strides = (C,) * 5

    def __del__(self):
        d = getattr(self, "desc", None)
        if d is not None:
            try:
                B.conv_norm_destroy(d)
            except Exception:
                pass

    def _tensor(self, t, dtype, rows, index, what):
        got, ld = rows_of(t, self.C, what)
        if t.dtype is not dtype or got != rows:
            raise ValueError(f"{what}: {got} rows of {t.dtype}, expected {rows} of {dtype}")
        if t.get_device() != index:
            raise ValueError(f"{what}: on another device than x")
        return t.data_ptr(), ld

    def _bind(self, x, index, rows, ldx, ldz, gate, x_out, h_out, want_x, stream):
        """Checks and allocates what a call needs besides x (on device index) and z, and gives
        the descriptor the strides: (x_out, h_out, addresses of gate, x_out, h_out and its
        scales)."""
        C, dtype, h_dtype, shape = self.C, self.dtype, self.h_dtype, x.shape
        if x.dtype is not dtype:
            raise ValueError(f"x: {x.dtype}, expected {dtype}")
        if self.index is not None and self.index != index:
            raise ValueError("x: on another device than the weights")
        gp = xop = hp = hsp = None
        ldg = ldxo = ldh = C
        if gate is not None:
            gp, ldg = self._tensor(gate, h_dtype, -(-rows // self.gate_rows), index, "gate")
        # of each output first the usual case: x's shape, contiguous
        if want_x:
            if x_out is None:
                with allocating_on(stream):
                    x_out = torch.empty(shape, dtype=dtype, device=x.device)
            if (x_out.dtype is dtype and x_out.is_contiguous() and x_out.shape == shape
                    and x_out.get_device() == index):
                xop = x_out.data_ptr()
            else:
                xop, ldxo = self._tensor(x_out, dtype, rows, index, "x_out")
        else:
            x_out = None
        if self.pre == B.CONV_NORM_NONE:
            h_out = None
        elif self.h_fmt is not None:
            if h_out is None:
                h_out = fp4.empty(rows, C, self.h_fmt, x.device, self.h_scale, stream)
            elif h_out.shape != (rows, C, self.h_fmt):
                raise ValueError("h_out: a 4-bit matrix of another shape or format")
            elif h_out.index != index:
                raise ValueError("h_out: on another device than x")
            h_out.tensor_scale = self.h_scale
            hp, hsp = h_out.codes_ptr, h_out.scales_ptr
        else:
            if h_out is None:
                with allocating_on(stream):
                    h_out = torch.empty(shape, dtype=h_dtype, device=x.device)
            if (h_out.dtype is h_dtype and h_out.is_contiguous() and h_out.shape == shape
                    and h_out.get_device() == index):
                hp = h_out.data_ptr()
            else:
                hp, ldh = self._tensor(h_out, h_dtype, rows, index, "h_out")
        strides = (ldx, ldz, ldg, ldxo, ldh)
        if strides != self._strides:
            B.conv_norm_set_strides(self.desc, *strides)
            self._strides = strides
        return x_out, h_out, gp, xop, hp, hsp

    def forward(self, x, z=None, gate=None, x_out=None, h_out=None, want_x=True, stream=None):
        """Returns (x', h).  x' is None when want_x is false, h when there is no norm_pre.
        x_out may be x itself."""
        with self._lock:
            C = self.C
            rows, ldx = rows_of(x, C, "x")
            index = x.get_device()
            handle = call_stream(index, stream)
            zp, ldz = None, C
            if z is not None:
                if (z.dtype is self.z_dtype and z.is_contiguous() and z.shape == x.shape
                        and z.get_device() == index):
                    zp = z.data_ptr()
                else:
                    zp, ldz = self._tensor(z, self.z_dtype, rows, index, "z")
            x_out, h_out, gp, xop, hp, hsp = self._bind(x, index, rows, ldx, ldz, gate, x_out,
                                                        h_out, want_x, stream)
            B.conv_norm_fwd(self.desc, rows, x.data_ptr(), zp, gp, xop, hp, hsp, handle)
            return x_out, h_out

    __call__ = forward
