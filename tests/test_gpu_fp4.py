"""Microscaled 4-bit quantisation (bit for bit against the definition) and the product
of 4-bit matrices (against 64 bits) on the GPU."""
import numpy as np
import pytest

from tests import fp4_ref as R
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu
FMTS = [R.MX, R.NV]
NAMES = {R.MX: "mx", R.NV: "nv"}


def _fp4():
    torch = need_gpu()
    from cnn_convolution_gemm_gb300 import fp4
    return torch, fp4


def _sync(torch):
    R.B.conv_sync_status(torch.cuda.current_stream().cuda_stream)


def _activations(rng, rows, cols):
    """Normal values of channel-wise different size, some exact ties and zeros among them."""
    x = rng.standard_normal((rows, cols)) * np.exp(0.7 * rng.standard_normal(cols))
    pick = rng.random((rows, cols))
    x = np.where(pick < 0.1, rng.choice([0.0, 0.25, -0.75, 1.25, 1.75, 2.5, -3.5, 5.0], (rows, cols)), x)
    x[rng.random(rows) < 0.1] = 0
    return x.astype(np.float32)


def _to(torch, a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def _f32(t):
    return t.float().cpu().numpy()


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 4096), (3, 16), (5, 31), (2, 33), (130, 64),
                                       (7, 100), (257, 272), (64, 1000), (33, 2080), (300, 129),
                                       (5000, 96), (2000, 200), (700, 5000)])
def test_quantize_is_the_definition(fmt, dtype, rows, cols):
    torch, fp4 = _fp4()
    rng = np.random.default_rng(rows * 10007 + cols)
    x = _to(torch, _activations(rng, rows, cols), getattr(torch, dtype))
    for g in ([1.0] if fmt == R.MX else [1.0, 0.01171875, 0.00873]):
        t = fp4.quantize(x, fmt, g)
        code, byte = R.quantize(_f32(x), fmt, g)
        got_code, got_byte = R.unpack(t)
        blocks = byte.shape[1]
        np.testing.assert_array_equal(got_byte[:, :blocks], byte)
        assert not got_byte[:, blocks:].any()
        n = min(code.shape[1], got_code.shape[1])
        # -0 and +0 stand for the same value
        np.testing.assert_array_equal(R.e2m1_value(got_code[:, :n]), R.e2m1_value(code[:, :n]))
        assert not got_code[:, cols:].any()
        y = fp4.dequantize(t, x.dtype)
        want = R.values(code, byte, fmt, cols, g)
        bits = 8 if dtype == "bfloat16" else 23
        np.testing.assert_allclose(y.double().cpu().numpy(), want, rtol=2.0 ** -bits, atol=0)


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
def test_quantize_extremes(fmt):
    """Infinities, NaNs, subnormals, the largest numbers: a NaN scale where a block is not
    finite, the definition elsewhere."""
    torch, fp4 = _fp4()
    rng = np.random.default_rng(1)
    x = rng.standard_normal((12, 96)).astype(np.float32)
    x[0, 3], x[1, 40], x[2, 95] = np.inf, np.nan, -np.inf
    x[3] *= np.float32(1e-38)
    x[4] = np.float32(1e-45) * rng.integers(-9, 9, 96)
    x[5] *= np.float32(3e37)
    x[6] = 0
    x[7] = np.where(rng.random(96) < 0.5, np.float32(3.3e38), np.float32(1.0))
    x[8] = -x[7]
    x[9] *= np.float32(1e-30)
    x[10, 5], x[10, 6] = -np.nan, np.inf
    for g in ([1.0] if fmt == R.MX else [1.0, 1e-30, 1e30, 3e-3]):
        t = fp4.quantize(torch.from_numpy(x).cuda(), fmt, g)
        code, byte = R.quantize(x, fmt, g)
        got_code, got_byte = R.unpack(t)
        np.testing.assert_array_equal(got_byte[:, : byte.shape[1]], byte)
        np.testing.assert_array_equal(R.e2m1_value(got_code), R.e2m1_value(code))
        y = fp4.dequantize(t, torch.float32).double().cpu().numpy()
        want = R.values(code, byte, fmt, 96, g)
        with np.errstate(over="ignore"):
            want = want.astype(np.float32).astype(np.float64)
        np.testing.assert_allclose(y, want, rtol=2.0 ** -23, atol=1e-45)


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
def test_every_code_and_scale_dequantizes(fmt):
    """All 16 codes under all scale bytes (but negative and NaN E4M3)."""
    torch, fp4 = _fp4()
    n_bytes = 255 if fmt == R.MX else 127
    b = R.BLOCK[fmt]
    code = np.tile(np.arange(16, dtype=np.uint8), (n_bytes, b // 16))
    byte = np.arange(n_bytes, dtype=np.uint8)[:, None]
    packed = R.pack_codes(code, b)
    t = fp4.empty(n_bytes, b, fmt, "cuda", 1.0 if fmt == R.MX else 0.25)
    t.codes.copy_(torch.from_numpy(packed).reshape(-1))
    R.B.conv_fp4_pack_scales(fmt, n_bytes, b, torch.from_numpy(byte).cuda().data_ptr(),
                             t.scales.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    y = fp4.dequantize(t, torch.float32).double().cpu().numpy()
    with np.errstate(over="ignore"):
        want = R.values(code, byte, fmt, b, t.tensor_scale).astype(np.float32)
    np.testing.assert_array_equal(y, want.astype(np.float64))


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
def test_quantize_strided_rows_and_offsets(fmt):
    """Rows inside a wider matrix, at addresses that allow no vector loads."""
    torch, fp4 = _fp4()
    rng = np.random.default_rng(2)
    wide = torch.from_numpy(_activations(rng, 37, 700)).cuda()
    for dt in (torch.bfloat16, torch.float32):
        w = wide.to(dt)
        for off, cols in ((1, 96), (3, 333), (8, 512), (0, 700)):
            x = w[:, off:off + cols]
            t = fp4.quantize(x, fmt)
            code, byte = R.quantize(_f32(x), fmt)
            got_code, got_byte = R.unpack(t)
            np.testing.assert_array_equal(got_byte[:, : byte.shape[1]], byte)
            np.testing.assert_array_equal(R.e2m1_value(got_code[:, :cols]),
                                          R.e2m1_value(code[:, :cols]))
            out = torch.full((37, 720), 7.0, dtype=dt, device="cuda")
            y = fp4.dequantize(t, out=out[:, 5:5 + cols])
            assert torch.equal(y, fp4.dequantize(t, dt))
            assert (out[:, :5] == 7).all() and (out[:, 5 + cols:] == 7).all()


# ---- product -------------------------------------------------------------------


def _product(fmt, M, C, K, x_dtype="bfloat16", y_dtype="bfloat16", act=0, bias=True, residual=False,
             seed=0, strided=False):
    torch, fp4 = _fp4()
    rng = np.random.default_rng(seed + 7 * M + 131 * C + 1009 * K + fmt)
    gx, gw, gy = (1.0, 1.0, 1.0) if fmt == R.MX else (0.0087, 0.0031 / np.sqrt(C), 0.0011)
    gx, gw, gy = (float(np.float32(v)) for v in (gx, gw, gy))
    xd = getattr(torch, x_dtype) if x_dtype else None
    yd = getattr(torch, y_dtype) if y_dtype else None
    x = _to(torch, _activations(rng, M, C), xd or torch.bfloat16)
    w = _to(torch, rng.standard_normal((K, C)) / np.sqrt(C), torch.bfloat16)
    b = _to(torch, 0.3 * rng.standard_normal(K), torch.float32) if bias else None
    r = _to(torch, rng.standard_normal((M, K)), yd) if residual else None
    out = None
    if strided:  # rows inside wider matrices
        x = torch.cat([x, x[:, :3]], 1)[:, :C]
        big = torch.full((M, K + 13), 7.0, dtype=yd, device="cuda")
        out = big[:, 5:5 + K]
        if residual:
            r = torch.cat([r, r[:, :1]], 1)[:, :K]
    layer = fp4.Fp4Linear(C, K, fmt, xd, yd, act, residual, gx, gy)
    layer.prepack(w, gw)
    xin = fp4.quantize(x, fmt, gx) if xd is None else x
    y = layer(xin, bias=b, residual=r, out=out)
    _sync(torch)
    xv = R.values(*R.quantize(_f32(x), fmt, gx), fmt, C, gx)
    wv = R.values(*R.quantize(_f32(w), fmt, gw), fmt, C, gw)
    pre = xv @ wv.T
    extra = np.zeros_like(pre)
    if bias:
        bb = b.double().cpu().numpy()
        pre, extra = pre + bb, extra + np.abs(bb)
    if residual:
        rr = r.double().cpu().numpy()
        pre, extra = pre + rr, extra + np.abs(rr)
    want = R.activate(pre, act)
    if yd is None:
        err = R.product_bound(xv, wv, want, extra, 24)
        R.check_quantized(y, want, err, fmt, gy)
        return y
    err = R.product_bound(xv, wv, want, extra, 8 if y_dtype == "bfloat16" else 24)
    got = y.double().cpu().numpy()
    assert got.shape == want.shape
    off = np.abs(got - want)
    assert (off <= err).all(), (off / err).max()
    if strided:
        assert (big[:, :5] == 7).all() and (big[:, 5 + K:] == 7).all()
    return y


SHAPES = [(1, 1, 1), (1, 32, 8), (1, 4096, 512), (2, 16, 31), (3, 33, 40), (7, 1000, 300),
          (8, 64, 32), (16, 2048, 1000), (17, 130, 129), (33, 256, 64), (64, 2048, 1000),
          (65, 512, 100), (100, 96, 257), (128, 256, 128), (129, 272, 384), (200, 64, 640),
          (255, 700, 255), (256, 1024, 256), (300, 1456, 1111), (515, 2080, 260), (777, 100, 520)]


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("M,C,K", SHAPES)
def test_product(fmt, M, C, K):
    _product(fmt, M, C, K)


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("M,C,K", [(1, 512, 256), (5, 100, 33), (64, 300, 1000), (300, 520, 400)])
@pytest.mark.parametrize("x,y,act,bias,residual", [
    ("float32", "float32", 0, False, False), ("bfloat16", "float32", 1, True, True),
    ("float32", "bfloat16", 2, True, True), ("bfloat16", "bfloat16", 3, False, True),
    (None, "float32", 4, True, False), (None, "bfloat16", 0, True, True),
    ("bfloat16", None, 3, True, False), (None, None, 0, False, False)])
def test_product_types_and_epilogues(fmt, M, C, K, x, y, act, bias, residual):
    _product(fmt, M, C, K, x, y, act, bias, residual)


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("M,C,K", [(3, 90, 70), (64, 320, 96), (140, 259, 301)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_product_strided_rows(fmt, M, C, K, dtype):
    _product(fmt, M, C, K, dtype, dtype, 1, True, True, strided=True)


# more tiles than the SMs take at once: 256 x 256 tiles over SM pairs, several to a pair; a
# second half of a pair's rows or columns that is empty, or up to 64 of 128; one and
# several k-steps
@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("M,C,K,x,y,act,bias,residual", [
    (2600, 1100, 1100, "bfloat16", "bfloat16", 1, True, True),
    (2600, 1100, 1104, None, "float32", 3, True, False),
    (5200, 64, 1025, "bfloat16", "bfloat16", 0, True, False),
    (4097, 200, 1300, "float32", "bfloat16", 4, False, True),
    (5250, 520, 1160, "bfloat16", None, 3, True, False),
    (3000, 272, 2096, None, None, 0, False, False),
    (2688, 2100, 1056, None, "float32", 2, True, True),
    (33, 96, 20000, "bfloat16", "bfloat16", 0, True, True)])
def test_product_of_many_tiles(fmt, M, C, K, x, y, act, bias, residual):
    _product(fmt, M, C, K, x, y, act, bias, residual)


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
def test_product_of_many_tiles_strided(fmt):
    _product(fmt, 2700, 1090, 1115, "bfloat16", "bfloat16", 1, True, True, strided=True)
    _product(fmt, 2700, 1090, 1115, "float32", "float32", 0, True, True, strided=True)


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9, 31, 32, 33, 40, 64, 65, 127, 160, 192])
@pytest.mark.parametrize("C,K", [(4500, 200), (1024, 1100)])
def test_product_of_few_rows(fmt, M, C, K):
    """Every way that rows are shared out, with the reduction split and whole."""
    _product(fmt, M, C, K, "bfloat16", "float32", 0, True, M % 2 == 0)


# long reductions of 2 to 72 tiles, shared out over as many CTAs as find room, evenly and
# not, and too short ones; empty blocks; a last k-step of one MMA
@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("M,C,K,x,y,act,bias,residual", [
    (65, 2048, 64, "bfloat16", "bfloat16", 0, True, True),
    (130, 3301, 201, "float32", "float32", 1, True, True),
    (300, 4500, 72, "bfloat16", None, 3, True, False),
    (257, 2600, 1000, None, None, 0, False, False),
    (140, 9000, 400, None, "bfloat16", 4, False, True),
    (129, 3090, 2100, "bfloat16", "float32", 2, True, False),
    (390, 4160, 1300, "bfloat16", "bfloat16", 1, False, True),
    (640, 5000, 512, "bfloat16", "bfloat16", 0, True, True), (520, 5200, 620, None, "float32", 3, True, False),
    (641, 5300, 641, "float32", None, 4, True, False), (700, 6210, 700, None, "bfloat16", 0, False, True),
    (768, 6500, 1024, "bfloat16", "float32", 1, True, True), (1000, 7600, 1100, None, None, 3, True, False)])
def test_product_of_split_reductions(fmt, M, C, K, x, y, act, bias, residual):
    _product(fmt, M, C, K, x, y, act, bias, residual)


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
def test_product_of_split_reductions_again(fmt):
    """The same bits every time, strided rows, and the output over the residual."""
    _product(fmt, 150, 4200, 203, "bfloat16", "bfloat16", 1, True, True, strided=True)
    torch, fp4 = _fp4()
    rng = np.random.default_rng(10)
    M, C, K = 200, 5000, 264
    x, r = _to(torch, _activations(rng, M, C), torch.bfloat16), _to(
        torch, rng.standard_normal((M, K)), torch.bfloat16)
    layer = fp4.Fp4Linear(C, K, fmt, has_residual=True)
    layer.prepack(_to(torch, rng.standard_normal((K, C)), torch.bfloat16))
    want = layer(x, residual=r)
    for _ in range(5):
        assert torch.equal(layer(x, residual=r), want)
    assert torch.equal(layer(x, residual=r, out=r), want)
    _sync(torch)


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("M,C,K", [(4, 256, 96), (150, 512, 300), (2600, 1100, 1100)])
def test_product_infinities_stay_in_their_rows(fmt, M, C, K):
    """A row of x that holds an Inf or a NaN gives a row of NaN; the other rows, and the
    rows of zeros, are untouched.  The same for a row of the weights and its column."""
    torch, fp4 = _fp4()
    rng = np.random.default_rng(5)
    x, w = rng.standard_normal((M, C)), rng.standard_normal((K, C))
    x[1] = 0
    clean = fp4.Fp4Linear(C, K, fmt)
    clean.prepack(_to(torch, w, torch.bfloat16))
    y0 = clean(_to(torch, x, torch.bfloat16))
    x[2, C // 2], w[K - 1, 3] = np.inf, np.nan
    layer = fp4.Fp4Linear(C, K, fmt)
    layer.prepack(_to(torch, w, torch.bfloat16))
    y = layer(_to(torch, x, torch.bfloat16))
    _sync(torch)
    assert torch.isnan(y[2]).all() and torch.isnan(y[:, K - 1]).all()
    keep = [i for i in range(M) if i != 2]
    assert torch.equal(y[keep][:, : K - 1], y0[keep][:, : K - 1])
    assert (y0[1] == 0).all()


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
def test_product_rows_do_not_depend_on_their_neighbours(fmt):
    """A row's result is the same bits alone and in any batch that takes the same kernel, and
    two runs give the same bits."""
    torch, fp4 = _fp4()
    rng = np.random.default_rng(6)
    C, K = 1024, 520
    x = _to(torch, _activations(rng, 600, C), torch.bfloat16)
    layer = fp4.Fp4Linear(C, K, fmt, y_dtype=torch.float32)
    layer.prepack(_to(torch, rng.standard_normal((K, C)), torch.bfloat16))
    y = layer(x)
    assert torch.equal(y, layer(x))
    assert torch.equal(y[200:], layer(x[200:]))
    wide = fp4.Fp4Linear(C, 3100, fmt, y_dtype=torch.float32)
    wide.prepack(_to(torch, rng.standard_normal((3100, C)), torch.bfloat16))
    xx = torch.cat([x] * 5)
    yy = wide(xx)
    assert torch.equal(yy, wide(xx)) and torch.equal(yy[:600], yy[2400:])
    small = layer(x[:9])
    assert torch.equal(small, layer(x[:9]))
    assert torch.equal(small[4:], layer(x[4:9]))


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("M,C,K", [(2, 192, 136), (200, 192, 136), (200, 192, 135), (2600, 1100, 1104)])
def test_product_into_its_residual(fmt, M, C, K):
    torch, fp4 = _fp4()
    rng = np.random.default_rng(8)
    x, r = _to(torch, _activations(rng, M, C), torch.bfloat16), _to(
        torch, rng.standard_normal((M, K)), torch.bfloat16)
    layer = fp4.Fp4Linear(C, K, fmt, has_residual=True)
    layer.prepack(_to(torch, rng.standard_normal((K, C)), torch.bfloat16))
    want = layer(x, residual=r)
    got = layer(x, residual=r, out=r)
    assert torch.equal(want, got)


def test_no_rows_and_other_streams():
    """Zero rows launch nothing; a layer used on two streams at once keeps them apart; a
    captured graph replays."""
    torch, fp4 = _fp4()
    B = R.B
    rng = np.random.default_rng(9)
    C, K = 256, 320
    layer = fp4.Fp4Linear(C, K, R.NV, x_scale=0.01)
    layer.prepack(_to(torch, rng.standard_normal((K, C)), torch.bfloat16), 0.001)
    n = B.conv_launch_count()
    assert layer(torch.empty(0, C, dtype=torch.bfloat16, device="cuda")).shape == (0, K)
    t = fp4.quantize(torch.empty(0, C, device="cuda"), R.MX)
    assert fp4.dequantize(t).shape == (0, C)
    assert B.conv_launch_count() == n
    xs = [_to(torch, _activations(rng, 150, C), torch.bfloat16) for _ in range(2)]
    want = [layer(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            got[i].append(layer(xs[i], stream=s.cuda_stream))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(want[i], y) for y in got[i])
    x = xs[0].clone()
    y = torch.empty(150, K, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        layer(x, out=y)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            layer(x, out=y)
    x.copy_(xs[1])
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want[1])


def test_offsets_past_32_bits():
    """Elements past 2^31 of x and y: the last rows of a tall matrix and of its product."""
    torch, fp4 = _fp4()
    M, C, K = 70000, 32768, 32
    x = torch.zeros(M, C, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(10)
    tail = _to(torch, _activations(rng, 5, C), torch.bfloat16)
    x[-5:] = tail
    layer = fp4.Fp4Linear(C, K, R.MX, y_dtype=torch.float32)
    layer.prepack(_to(torch, rng.standard_normal((K, C)), torch.bfloat16))
    y = layer(x)
    xv = R.values(*R.quantize(_f32(tail), R.MX), R.MX, C)
    wv = R.tensor_values(layer.w)
    want = xv @ wv.T
    err = R.product_bound(xv, wv, want, 0, 24)
    assert (np.abs(y[-5:].double().cpu().numpy() - want) <= err).all()
    assert not y[:-5].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [23, 300, 1001, 1536, 2420])
def test_quantize_at_every_alignment(dtype, cols):
    """Rows that start anywhere: the codes of aligned rows, and values that go back to their
    places and no others."""
    torch, fp4 = _fp4()
    torch.manual_seed(cols)
    dt, rows = (torch.bfloat16 if dtype == "bf16" else torch.float32), 21
    wide = torch.zeros(rows, -(-cols // 16) * 16, dtype=dt, device="cuda")
    wide[:, :cols] = torch.randn(rows, cols, device="cuda").to(dt)
    for fmt, g in ((R.MX, 1.0), (R.NV, 0.003)):
        want = fp4.quantize(wide[:, :cols], fmt, g)
        blocks = -(-cols // R.BLOCK[fmt])
        scales = R.unpack(want)[1][:, :blocks]
        values = fp4.dequantize(want, dtype=dt, out=torch.empty_like(wide)[:, :cols])
        for offset in range(9):
            for ld in (cols, cols + 1, cols + 5):
                buf = torch.full((offset + rows * ld + 9,), 7.5, dtype=dt, device="cuda")
                at = buf.as_strided((rows, cols), (ld, 1), offset)
                at.copy_(wide[:, :cols])
                got = fp4.quantize(at, fmt, g)
                assert torch.equal(got.codes, want.codes)
                np.testing.assert_array_equal(R.unpack(got)[1][:, :blocks], scales)
                buf.fill_(7.5)
                fp4.dequantize(got, out=at)
                assert torch.equal(at, values)
                at.fill_(7.5)
                assert bool((buf == 7.5).all())


def _at_16_of_32(torch, n):
    """n bytes at an address that is a multiple of 16, not of 32, and the buffer around them."""
    buf = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    start = 16 + -buf.data_ptr() % 32
    return buf, buf[start:start + n], start


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("M,C,K", [(3000, 272, 2096), (2600, 256, 2112), (130, 96, 192), (5, 300, 64)])
def test_product_into_codes_at_16_bytes(fmt, M, C, K):
    """4-bit outputs need 16-byte alignment only: rows of whole 32-byte pieces that start
    between two of them, in the tiles of both sizes and in the kernel for few rows."""
    torch, fp4 = _fp4()
    rng = np.random.default_rng(M)
    layer = fp4.Fp4Linear(C, K, fmt, y_dtype=None, act=R.B.CONV_ACT_RELU)
    layer.prepack(_to(torch, rng.standard_normal((K, C)), torch.bfloat16))
    x = _to(torch, _activations(rng, M, C), torch.bfloat16)
    want = layer(x)
    cb, sb = R.B.conv_fp4_size(fmt, M, K)
    cbuf, codes, c0 = _at_16_of_32(torch, cb)
    sbuf, scales, s0 = _at_16_of_32(torch, sb)
    got = layer(x, out=fp4.Fp4Tensor(M, K, fmt, 1.0, codes, scales))
    _sync(torch)
    assert got.codes_ptr % 32 == 16 and torch.equal(codes, want.codes)
    np.testing.assert_array_equal(R.unpack(got)[1], R.unpack(want)[1])
    for buf, at, n in ((cbuf, c0, cb), (sbuf, s0, sb)):
        assert (buf[:at] == 0xA5).all() and (buf[at + n:] == 0xA5).all()


@pytest.mark.parametrize("what", ["layer", "block"])
def test_graphs_keep_their_workspaces(what):
    """A graph of few rows replays to the same bits after the layer served more rows on the same
    stream and other tensors took what that freed; and leaves those tensors alone."""
    torch, fp4 = _fp4()
    from cnn_convolution_gemm_gb300.residual_block import Fp4ResidualBlock
    rng = np.random.default_rng(11)
    C, K = 256, 320
    if what == "layer":
        layer = fp4.Fp4Linear(C, K, R.MX)
        layer.prepack(_to(torch, rng.standard_normal((K, C)), torch.bfloat16))
        call = layer
    else:
        layer = Fp4ResidualBlock(C, K, R.MX)
        layer.prepack(_to(torch, rng.standard_normal((K, C)), torch.bfloat16),
                      _to(torch, rng.standard_normal((C, K)), torch.bfloat16))
        call = lambda x: layer(x)[1]  # noqa: E731
    x = _to(torch, _activations(rng, 40, C), torch.bfloat16)
    many = _to(torch, _activations(rng, 3000, C), torch.bfloat16)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        want = call(x).clone()
        side.synchronize()
        graphs, outs = [], []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                outs.append(call(x))
            graphs.append(g)
        call(many)
        taken = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda")
                 for n in (512, 4096, 8192, 16384, 1 << 20) for _ in range(64)]
        for _ in range(3):
            for g, out in zip(graphs, outs):
                out.zero_()
                g.replay()
                call(many)
        side.synchronize()
    for out in outs:
        assert torch.equal(out, want)
    assert all(bool((t == 0x5A).all()) for t in taken)


def _activation_case(act, M, K, y_dtype, fmt, bound):
    """act of known values, which a product of zeros takes from its bias: outputs within bound(v,
    result) of the result (and 1e-35, where fp32 cannot hold it in full), then rounded to y's type.
    Infinities and NaN give what the definition's arithmetic gives, in their columns alone (4
    bits: a NaN scale for their block)."""
    torch, fp4 = _fp4()
    rng = np.random.default_rng(act)
    C, n = 64, K - 64
    v = np.concatenate([np.linspace(-14, 14, n - n // 4), -np.exp(rng.uniform(-20, 5, n // 8)),
                        np.exp(rng.uniform(-20, 5, n // 4 - n // 8)), np.zeros(64)]).astype(np.float32)
    special = np.array([np.inf, -np.inf, np.nan, -np.nan, 3e38, -3e38, 0.0, -0.0], np.float32)
    v[n + 5:n + 13] = special
    if y_dtype is None:
        v[n:] = np.where(np.isfinite(v[n:]), v[n:], 0)  # a second run has them
    layer = fp4.Fp4Linear(C, K, fmt, y_dtype=getattr(torch, y_dtype) if y_dtype else None, act=act)
    layer.prepack(_to(torch, rng.standard_normal((K, C)), torch.bfloat16))
    x = torch.zeros(M, C, dtype=torch.bfloat16, device="cuda")
    y = layer(x, bias=torch.from_numpy(v).cuda())
    _sync(torch)
    d = v.astype(np.float64)
    with np.errstate(all="ignore"):
        if act == R.B.CONV_ACT_GELU:
            from scipy.special import ndtr
            want = d * ndtr(d)
        elif act == R.B.CONV_ACT_SILU:
            want = d / (1 + np.exp(-d))
        else:
            want = R.activate(d, act)
        err = bound(np.clip(d, -1e3, 1e3), np.abs(want)) + 1e-35
    if y_dtype is None:
        keep = slice(0, min(M, 130))
        part = fp4.Fp4Tensor(y.rows, K, fmt, 1.0, y.codes, y.scales)
        R.check_quantized(part, np.tile(want, (M, 1)), np.tile(err, (M, 1)), fmt, 1.0)
        v[n + 5:n + 8] = special[:3]
        bad = layer(x, bias=torch.from_numpy(v).cuda())
        _sync(torch)
        code, byte = R.unpack(bad)
        code0, byte0 = R.unpack(y)
        b, nan = R.BLOCK[fmt], 0xFF if fmt == R.MX else 0x7F
        blocks = n // b  # of the values before the special ones
        np.testing.assert_array_equal(byte[:, :blocks], byte0[:, :blocks])
        np.testing.assert_array_equal(code[:, :n], code0[:, :n])
        # relu6 leaves the first infinity finite; a NaN stays
        assert (byte[keep, blocks] == nan).all() and not code[:, n:n + b].any()
        return
    got = y.double().cpu().numpy()
    odd = ~np.isfinite(want)
    np.testing.assert_array_equal(got[:, odd], np.tile(want[odd], (M, 1)))
    off = np.abs(got[:, ~odd] - want[~odd])
    limit = err[~odd] + R.half_spacing(np.abs(want[~odd]) + err[~odd], y_dtype)
    assert (off <= limit).all(), (off / limit).max()


# one row, the tiles of both sizes
ACT_SHAPES = [(3, 1088), (130, 1088), (2600, 2112)]


def _gelu_bound(v, want, y_dtype):
    """fp32 outputs, in units of 2^-23 of the result: the polynomial 1, that evaluated 4,
    1 / (1 + p |x|) and how the polynomial goes with it 4, the exponential 2 and its argument's
    rounding 0.6 x^2, products 2.  Others: 4.2e-7 (0.75e-7 of Phi from the polynomial, the rest
    roundings), and what the polynomial is off by relatively above -3 and -5."""
    if y_dtype == "float32":
        return want * (v * v + 14) * 2.0 ** -23
    rel = np.where(v > -3, 6e-5, np.where(v > -5, 2e-3, np.inf))
    with np.errstate(invalid="ignore"):
        return np.fmin(4.2e-7, np.where(np.isinf(rel), np.inf, want * np.where(np.isinf(rel), 0, rel)))


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("y_dtype", ["float32", "bfloat16", None])
@pytest.mark.parametrize("M,K", ACT_SHAPES)
def test_gelu_values(M, K, y_dtype, fmt):
    _activation_case(R.B.CONV_ACT_GELU, M, K, y_dtype, fmt, lambda v, w: _gelu_bound(v, w, y_dtype))


@pytest.mark.parametrize("act", [R.B.CONV_ACT_NONE, R.B.CONV_ACT_RELU, R.B.CONV_ACT_RELU6])
@pytest.mark.parametrize("y_dtype", ["float32", "bfloat16", None])
@pytest.mark.parametrize("M,K", ACT_SHAPES)
def test_exact_activations_values(M, K, y_dtype, act):
    _activation_case(act, M, K, y_dtype, R.NV, lambda v, w: 0.0 * v)


@pytest.mark.parametrize("fmt", FMTS, ids=NAMES.get)
@pytest.mark.parametrize("y_dtype", ["float32", "bfloat16", None])
@pytest.mark.parametrize("M,K", ACT_SHAPES)
def test_silu_values(M, K, y_dtype, fmt):
    """In units of 2^-23 of the result.  fp32 outputs: exp 2, 1 + exp and the product 0.5 each,
    the reciprocal 1.  Others: exp2 2 and its argument's rounding 0.75 |x| instead."""
    exp = (lambda v: 2.0) if y_dtype == "float32" else (lambda v: 2 + 0.75 * np.abs(v))
    _activation_case(R.B.CONV_ACT_SILU, M, K, y_dtype, fmt, lambda v, w: w * (exp(v) + 2) * 2.0 ** -23)
