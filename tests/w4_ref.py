"""References in 64 bits (numpy) of the 8-bit matrices and of the products with integer 4-bit
weights, from their definitions in gbconv.h."""
import math

import numpy as np

E4M3, INT8 = 0, 1
TOP = {E4M3: 448.0, INT8: 127.0}
NAMES = {E4M3: "e4m3", INT8: "int8"}


def e4m3_values():
    """The values of the 256 E4M3 bytes."""
    v = np.zeros(256)
    for b in range(128):
        e, f = b >> 3, b & 7
        v[b] = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
    v[127] = np.nan
    v[128:] = -v[:128]
    return v


def code_values(byte, fmt):
    return e4m3_values()[byte] if fmt == E4M3 else byte.astype(np.int8).astype(np.float64)


def levels(fmt):
    return e4m3_values()[:127] if fmt == E4M3 else np.arange(128.0)


def _groups(x, group):
    rows, cols = x.shape
    g = group or cols
    padded = np.zeros((rows, -(-cols // g) * g))
    padded[:, :cols] = x
    return padded.reshape(rows, -1, g)


def scales(x, fmt, group):
    """[rows][groups] fp32; NaN where a group is not finite."""
    top = np.abs(_groups(x.astype(np.float64), group)).max(axis=2)
    s = np.maximum((np.where(np.isfinite(top), top, 0) / TOP[fmt]).astype(np.float32),
                   np.float32(2.0 ** -100))
    return np.where(np.isfinite(top), s, np.float32(np.nan))


def quantize(x, fmt, group):
    """(values of the codes [rows][cols], scales [rows][groups]).  The nearest code is found by
    exact comparisons: |x| with (a + b) / 2 * s, a product of at most 9 and 24 bits."""
    cols = x.shape[1]
    s = scales(x, fmt, group)
    v = _groups(x.astype(np.float64), group)
    lv = levels(fmt)
    mid = (lv[1:] + lv[:-1]) / 2
    code = np.zeros(v.shape)
    for r in range(v.shape[0]):
        for g in range(v.shape[1]):
            if np.isfinite(s[r, g]):
                a, at = np.abs(v[r, g]), mid * float(s[r, g])
                lo, hi = np.searchsorted(at, a, "left"), np.searchsorted(at, a, "right")
                code[r, g] = np.copysign(lv[np.where((lo != hi) & (hi % 2 == 1), lo, hi)], v[r, g])
    return code.reshape(len(x), -1)[:, :cols], s


def values(code, s, group):
    cols = code.shape[1]
    return code * np.repeat(s.astype(np.float64), group or cols, axis=1)[:, :cols]


def pack_weights(q):
    """uint8 [K][ceil(C / 2)]."""
    q = np.pad(q, ((0, 0), (0, q.shape[1] % 2)))
    return (q[:, 0::2] | (q[:, 1::2] << 4)).astype(np.uint8)


def weights(q, scale, zero, group):
    """(code - zero) * scale in 64 bits; zero None: 8."""
    C = q.shape[1]

    def over(t):
        return np.repeat(t.astype(np.float64), group or C, axis=1)[:, :C]

    return (q - (8.0 if zero is None else over(zero))) * over(scale)


_erf = np.vectorize(math.erf, otypes=[float])


def act(v, kind):
    """binding.CONV_ACT_* in 64 bits."""
    if kind == 3:
        return 0.5 * v * (1 + _erf(v * math.sqrt(0.5)))
    with np.errstate(over="ignore"):
        return (v, np.maximum(v, 0), np.clip(v, 0, 6), None,
                v / (1 + np.exp(-v)))[kind]
