"""A residual block in 4 bits (conv_fp4_block_* of gbconv.h): two fully connected layers
(1x1 convolutions over NHWC pixels) between the norms around them.

  h  = norm_pre(x), 4 bits             one pass over x
  t  = gelu(h W1^T + b1), 4 bits       quantised in the product's epilogue
  z  = t W2^T + b2
  x' = x + residual_scale * g(gate) * norm_post(z);  h' = norm_next(x')    one pass

h' is what the next block starts from: blocks chained with ``chain=True`` hand it on in
4 bits, so the stream x is read and written once per block.
"""
from __future__ import annotations

import torch

from . import binding as B
from . import fp4
from .fp4 import Fp4Linear
from .norm import ResidualNorm


class Fp4ResidualBlock:
    """RMS norms throughout; gate, gate_rows, residual_scale as in ``ResidualNorm``.  dtype: of
    x, gate, x' and h'; z, between the second layer and the norm behind it, is fp32.
    w_next: weight of the norm behind the block (the next block's, or the final one);
    chain: give h' in 4 bits with tensor scale next_scale instead of dtype.
    h_scale, t_scale: tensor scales of h and t (CONV_FP4_NV).  Threads may share a block and
    its parts."""

    def __init__(self, C, hidden, fmt=B.CONV_FP4_MX, dtype=torch.bfloat16, eps=1e-6,
                 residual_scale=1.0, gate=B.CONV_GATE_NONE, gate_rows=1, w_pre=None, w_post=None,
                 w_next=None, b1=None, b2=None, h_scale=1.0, t_scale=1.0, chain=False,
                 next_scale=1.0):
        self.C, self.hidden, self.fmt, self.dtype = C, hidden, fmt, dtype
        self.h_scale, self.t_scale = h_scale, t_scale
        for b, n in ((b1, hidden), (b2, C)):
            if b is not None and (b.dtype != torch.float32 or b.numel() != n
                                  or not b.is_contiguous()):
                raise ValueError("b1, b2: expected contiguous fp32 [hidden], [C]")
            if b is not None and b.get_device() < 0:
                raise ValueError("b1, b2: must be on the GPU")
        self.b1, self.b2 = b1, b2
        self.norm_in = ResidualNorm(C, dtype, eps=eps, pre=B.CONV_NORM_RMS,
                                    w_pre=w_pre, h_fmt=fmt, h_scale=h_scale)
        self.fc1 = Fp4Linear(C, hidden, fmt, x_dtype=None, y_dtype=None, act=B.CONV_ACT_GELU,
                             x_scale=h_scale, y_scale=t_scale)
        self.fc2 = Fp4Linear(hidden, C, fmt, x_dtype=None, y_dtype=torch.float32, x_scale=t_scale)
        self.norm_out = ResidualNorm(C, dtype, torch.float32, eps=eps, post=B.CONV_NORM_RMS,
                                     w_post=w_post, pre=B.CONV_NORM_RMS, w_pre=w_next, gate=gate,
                                     gate_rows=gate_rows, residual_scale=residual_scale,
                                     h_fmt=fmt if chain else None, h_scale=next_scale,
                                     h_dtype=dtype)
        self.desc = B.conv_fp4_block_create(self.norm_in.desc, self.fc1.desc, self.fc2.desc,
                                            self.norm_out.desc)
        # one lock for the descriptors, which the parts' own calls change too
        self._lock = self.norm_in._lock
        for part in (self.fc1, self.fc2, self.norm_out):
            part._lock = self._lock
        self._held = (None, None)  # the weights that desc has the addresses of
        self._sizes, self._ws = {}, fp4.Workspaces()  # sizes: rows -> workspace bytes

    def __del__(self):
        d = getattr(self, "desc", None)
        if d is not None:
            try:
                B.conv_fp4_block_destroy(d)
            except Exception:
                pass

    def prepack(self, w1, w2, w1_scale=1.0, w2_scale=1.0, stream=None):
        """Quantise the weights w1 [hidden][C], w2 [C][hidden] once."""
        self.fc1.prepack(w1, w1_scale, stream)
        self.fc2.prepack(w2, w2_scale, stream)

    def load(self, w1, s1, g1, w2, s2, g2, stream=None):
        """Weights held in 4 bits (codes, row-by-row scales, tensor scale of each)."""
        self.fc1.load(w1, s1, g1, stream)
        self.fc2.load(w2, s2, g2, stream)

    def _hold(self, w1, w2):
        if w1 is None or w2 is None:
            raise RuntimeError("prepack() or load() the weights first")
        held = (w1.index, w2.index, self.norm_in.index, self.norm_out.index,
                *(b.get_device() for b in (self.b1, self.b2) if b is not None))
        if set(held) - {None, w1.index}:
            raise ValueError("weights and biases: on different devices")
        b1, b2 = (None if b is None else b.data_ptr() for b in (self.b1, self.b2))
        B.conv_fp4_block_set_weights(self.desc, w1.codes_ptr, w1.scales_ptr, b1, w2.codes_ptr,
                                     w2.scales_ptr, b2)
        self._held = (w1, w2)

    def forward(self, x, gate=None, h=None, x_out=None, h_out=None, stream=None):
        """x [..., C] -> (x', h').  h: norm_pre(x) in 4 bits when the block before handed
        it on, else None."""
        with self._lock:
            C, norm_in, fc2 = self.C, self.norm_in, self.fc2
            w1, w2 = self.fc1.w, fc2.w
            if w1 is None or (w1, w2) != self._held:
                self._hold(w1, w2)
            rows, ldx = fp4.rows_of(x, C, "x")
            index = w1.index
            handle = fp4.call_stream(index, stream)
            if x.get_device() != index:
                raise ValueError("x: on another device than the weights")
            hp = hsp = None
            if h is not None:
                if (h.shape, h.tensor_scale) != ((rows, C, self.fmt), self.h_scale):
                    raise ValueError("h: a 4-bit matrix of another shape, format or tensor scale")
                if h.index != index:
                    raise ValueError("h: on another device than the weights")
                hp, hsp = h.codes_ptr, h.scales_ptr
            x_out, h_out, gp, xop, hop, hosp = self.norm_out._bind(
                x, index, rows, ldx, C, gate, x_out, h_out, True, stream)
            # the strides of the block's own calls: those of a part's own call stay in its descriptor
            if norm_in._strides != (ldx, C, C, C, C):
                norm_in._strides = (ldx, C, C, C, C)
                B.conv_norm_set_strides(norm_in.desc, *norm_in._strides)
            if fc2._strides != (self.hidden, C, C):
                fc2._strides = (self.hidden, C, C)
                B.conv_fp4_set_strides(fc2.desc, *fc2._strides)
            need = self._sizes.get(rows)
            if need is None:
                need = self._sizes[rows] = B.conv_fp4_block_workspace_size(self.desc, rows)
            # held until the launches are enqueued
            ws = self._ws.get(need, w1.device, index, stream, handle) if need else None
            B.conv_fp4_block_fwd(self.desc, rows, x.data_ptr(), hp, hsp, gp, xop, hop, hosp,
                                 ws.data_ptr() if need else None, need, handle)
            return x_out, h_out

    __call__ = forward
