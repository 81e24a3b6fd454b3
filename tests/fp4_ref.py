"""The microscaled 4-bit formats, their product and the norms around a block in plain
numpy: codes and scales from the definitions (bit for bit), everything else in 64 bits."""
import numpy as np

from cnn_convolution_gemm_gb300 import binding as B

MX, NV = B.CONV_FP4_MX, B.CONV_FP4_NV
BLOCK = {MX: 32, NV: 16}
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# between code i and i + 1; a tie goes to the even code
MIDDLES = (LEVELS[:-1] + LEVELS[1:]) / 2


def e2m1_code(v):
    """Codes of finite float values: nearest level, ties to even, saturating."""
    a = np.abs(np.asarray(v, np.float64))
    code = np.zeros(a.shape, np.uint8)
    for i, m in enumerate(MIDDLES):
        code += (a > m) if i % 2 == 0 else (a >= m)
    return code | (np.signbit(v).astype(np.uint8) << 3)


def e2m1_value(code):
    v = LEVELS[code & 7]
    return np.where(code & 8, -v, v)


def e4m3_value(byte):
    byte = np.asarray(byte, np.int64)
    e, f = (byte >> 3) & 15, byte & 7
    v = np.where(e > 0, np.ldexp(1 + f / 8, e - 7), np.ldexp(f / 8, -6))
    return np.where((byte & 0x7F) == 0x7F, np.nan, v)


E4M3 = e4m3_value(np.arange(127))  # 0 .. 448, increasing


def e4m3_byte(v):
    """Nearest E4M3 byte of values in [0, 448], ties to the even byte."""
    v = np.asarray(v, np.float64)
    hi = np.clip(np.searchsorted(E4M3, v, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    mid = (E4M3[hi] + E4M3[lo]) / 2
    up = (v > mid) | ((v == mid) & (hi % 2 == 0))
    return np.where(v >= E4M3[hi], hi, np.where(up, hi, lo)).astype(np.uint8)


def quantize(x, fmt, g=1.0):
    """x [rows, cols] float32 -> (codes [rows, blocks * block], scale bytes [rows, blocks])."""
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    b = BLOCK[fmt]
    blocks = -(-cols // b)
    full = np.zeros((rows, blocks * b), np.float32)
    full[:, :cols] = x
    v = full.reshape(rows, blocks, b)
    bad = ~np.isfinite(v).all(axis=2)
    v = np.where(bad[:, :, None], np.float32(0), v)
    top = np.abs(v).max(axis=2)
    g = np.float32(g)
    with np.errstate(all="ignore"):
        if fmt == MX:
            _, e = np.frexp(top.astype(np.float64))
            e = np.where(top > 0, np.maximum(e - 3, -127), -127)
            byte = (e + 127).astype(np.uint8)
            q = np.ldexp(v.astype(np.float64), -e[:, :, None])
        else:
            byte = e4m3_byte(np.minimum(top / (np.float32(6) * g), np.float32(448)))
            t = (e4m3_value(byte).astype(np.float32) * g)[:, :, None]
            q = np.where(t > 0, (v / np.where(t > 0, t, 1)).astype(np.float32), 0)
    code = np.where(bad[:, :, None], 0, e2m1_code(q))
    if fmt == NV:
        code = np.where(byte[:, :, None] == 0, 0, code)
    byte = np.where(bad, 0xFF if fmt == MX else 0x7F, byte).astype(np.uint8)
    return code.reshape(rows, -1).astype(np.uint8), byte


def scale_values(byte, fmt, g=1.0):
    if fmt == MX:
        v = np.ldexp(1.0, byte.astype(np.int64) - 127)
        return np.where(byte == 255, np.nan, v)
    return e4m3_value(byte) * np.float64(np.float32(g))


def values(code, byte, fmt, cols, g=1.0):
    s = np.repeat(scale_values(byte, fmt, g), BLOCK[fmt], axis=1)
    with np.errstate(invalid="ignore"):
        return (e2m1_value(code) * s)[:, :cols]


def pack_codes(code, cols):
    """[rows, 16 * ceil(cols / 32)] bytes as the library holds them."""
    rows = code.shape[0]
    full = np.zeros((rows, 32 * -(-cols // 32)), np.uint8)
    full[:, : code.shape[1]] = code[:, : full.shape[1]]
    return (full[:, 0::2] | (full[:, 1::2] << 4)).astype(np.uint8)


def tiled_index(rows, blocks, tiles):
    """Byte offsets of the scales [rows, blocks] in the tiled order."""
    r = np.arange(rows)[:, None]
    b = np.arange(blocks)[None, :]
    return ((r // 128) * tiles + b // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4


def tiles_per_row(fmt, cols):
    return -(-cols // (4 * BLOCK[fmt]))


def unpack(t):
    """(codes [rows, pitch * 2], scale bytes [rows, 4 * tiles]) of an Fp4Tensor on the GPU."""
    packed = t.codes.cpu().numpy().reshape(t.rows, -1)
    code = np.empty((t.rows, packed.shape[1] * 2), np.uint8)
    code[:, 0::2], code[:, 1::2] = packed & 15, packed >> 4
    tiles = tiles_per_row(t.fmt, t.cols)
    return code, t.scales.cpu().numpy()[tiled_index(t.rows, 4 * tiles, tiles)]


def tensor_values(t):
    """The float64 values of an Fp4Tensor on the GPU."""
    code, byte = unpack(t)
    b = BLOCK[t.fmt]
    blocks = -(-t.cols // b)
    full = np.zeros((t.rows, blocks * b), np.uint8)
    n = min(full.shape[1], code.shape[1])
    full[:, :n] = code[:, :n]
    return values(full, byte[:, :blocks], t.fmt, t.cols, t.tensor_scale)


def activate(v, act):
    from scipy.special import erf
    with np.errstate(over="ignore"):
        if act == B.CONV_ACT_RELU:
            return np.where(v < 0, 0, v)
        if act == B.CONV_ACT_RELU6:
            return np.where(v < 0, 0, np.where(v > 6, 6, v))
        if act == B.CONV_ACT_GELU:
            return 0.5 * v * (1 + erf(v / np.sqrt(2)))
        if act == B.CONV_ACT_SILU:
            return v / (1 + np.exp(-v))
    return v


def norm(v, kind, eps, w=None, b=None):
    if kind == B.CONV_NORM_NONE:
        return v
    mean = v.mean(axis=1, keepdims=True) if kind == B.CONV_NORM_LAYER else 0.0
    out = (v - mean) / np.sqrt(((v - mean) ** 2).mean(axis=1, keepdims=True) + eps)
    out = out if w is None else out * w
    return out if b is None else out + b


def product_bound(xv, wv, y, extra, out_bits):
    """How far a product may be from 64 bits.  Each of the C / 64 + 1 accumulation steps
    adds 64 exact products to an fp32 sum, aligned to the largest of them: at most
    2^-22 of the sum of magnitudes a step, with 8 steps more for joining split sums;
    the epilogue (scale, bias, residual, activation, whose slope is below 1.13)
    rounds a handful of times; then one rounding to the output's bits."""
    steps = xv.shape[1] / 64 + 9
    size = np.abs(np.nan_to_num(xv)) @ np.abs(np.nan_to_num(wv)).T
    return 1.13 * (steps * 2.0 ** -22 * size + 2.0 ** -21 * (size + extra)) + (
        2.0 ** -out_bits * np.abs(y)) + 1e-37


def check_quantized(t, y, err, fmt, g):
    """An Fp4Tensor made from values within err of y: every scale is one that a largest
    magnitude within err gives, and every value is nearest to y but for err and the quotient's rounding."""
    code, byte = unpack(t)
    b = BLOCK[fmt]
    rows, cols = y.shape
    blocks = -(-cols // b)
    full_y, full_e = np.zeros((rows, blocks * b)), np.zeros((rows, blocks * b))
    full_y[:, :cols], full_e[:, :cols] = y, err
    yb, eb = full_y.reshape(rows, blocks, b), full_e.reshape(rows, blocks, b)
    lo = np.maximum(np.abs(yb) - eb, 0).max(axis=2)
    hi = (np.abs(yb) + eb).max(axis=2)
    bytes_of = lambda top: quantize(np.repeat(top.reshape(-1, 1), b, 1), fmt, g)[1].reshape(rows, blocks)  # noqa: E731
    got = byte[:, :blocks].astype(int)
    assert (bytes_of(lo * (1 - 1e-6)) <= got).all() and (got <= bytes_of(hi * (1 + 1e-6))).all()
    assert (byte[:, blocks:] == 0).all() and (code[:, cols:] == 0).all()
    s = scale_values(byte[:, :blocks], fmt, g)[:, :, None]
    n = code.shape[1]
    full_c = np.zeros((rows, blocks * b), np.uint8)
    full_c[:, : min(n, blocks * b)] = code[:, : blocks * b]
    full_c = full_c.reshape(rows, blocks, b)
    mag = full_c & 7
    v = e2m1_value(full_c) * s
    below = np.where(mag > 0, LEVELS[mag] - LEVELS[np.maximum(mag, 1) - 1], 1.0) / 2
    above = np.where(mag < 7, LEVELS[np.minimum(mag, 6) + 1] - LEVELS[mag], np.inf) / 2
    away = np.abs(yb) - np.abs(v)
    slack = eb + 1e-6 * np.abs(yb)
    # above 6 the value saturates; a scale of 0 (NV) holds nothing but zeros
    far = np.where(s > 0, np.nan_to_num(above * np.where(s > 0, s, 1), posinf=np.inf), np.inf)
    assert (away <= far + slack).all()
    assert (-away <= below * s + slack).all()
    wrong = (np.sign(v) * np.sign(yb) < 0) & (np.abs(v) > 0) & (np.abs(yb) > slack)
    assert not wrong.any()


def half_spacing(v, dt):
    """The most that one rounding to dt moves a value of up to this magnitude: half the distance of
    its neighbours, of 8 or 24 significant bits."""
    return np.ldexp(1.0, np.frexp(v + 1e-37)[1] - {"bfloat16": 9, "float32": 25}[dt])
