"""8-bit matrices with scales: bit for bit against the definition, and the norms that give them
against 64 bits, on the GPU."""
import numpy as np
import pytest

from tests import w4_ref as R
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu
FMTS = [R.E4M3, R.INT8]


def _q8():
    torch = need_gpu()
    from cnn_convolution_gemm_gb300 import q8
    return torch, q8


def _sync(torch):
    from cnn_convolution_gemm_gb300 import binding as B
    B.conv_sync_status(torch.cuda.current_stream().cuda_stream)


def _activations(rng, rows, cols):
    """Values of channel-wise different size, some of them ties or next to ties of their row's
    scale (halves and quarters of its largest), zeros and rows of zeros."""
    x = rng.standard_normal((rows, cols)) * np.exp(0.7 * rng.standard_normal(cols))
    top = np.abs(x).max(axis=1, keepdims=True)
    pick = rng.random((rows, cols))
    x = np.where(pick < 0.1, top * rng.choice([0.5, -0.25, 0.5 / 448, 17 / 448, -19 / 448,
                                               1.5 / 127, 2.5 / 127], (rows, cols)), x)
    x[pick > 0.95] = 0
    x[rng.random(rows) < 0.1] = 0
    return x.astype(np.float32)


def _f32(t):
    return t.float().cpu().numpy()


def unpack(t):
    """(values of the codes [rows][cols], padding bytes, scales [rows][groups])."""
    pitch = 16 * -(-t.cols // 16)
    byte = t.codes[: t.rows * pitch].view(t.rows, pitch).cpu().numpy()
    groups = -(-t.cols // 128) if t.group else 1
    s = t.scales[: t.rows * groups].view(t.rows, groups).cpu().numpy()
    return R.code_values(byte[:, : t.cols], t.fmt), byte[:, t.cols:], s


def _check(q8, torch, x, fmt, group, t=None):
    t = q8.quantize(x, fmt, group) if t is None else t
    code, s = R.quantize(_f32(x).reshape(-1, x.shape[-1]), fmt, group)
    got, pad, got_s = unpack(t)
    np.testing.assert_array_equal(got_s, s)
    np.testing.assert_array_equal(got, code)  # -0 and +0 stand for the same value
    assert not pad.any()
    for dtype in (torch.bfloat16, torch.float32):
        want = torch.from_numpy(R.values(code, s, group)).to(torch.float32).to(dtype)
        y = q8.dequantize(t, dtype).cpu()
        assert torch.equal(torch.nan_to_num(y, 7.0), torch.nan_to_num(want, 7.0))


SIZES = [(1, 1), (1, 4096), (3, 16), (5, 31), (2, 33), (130, 64), (7, 100), (67, 128), (65, 129),
         (257, 272), (64, 1000), (33, 2080), (300, 250), (3000, 96), (41, 513), (9, 5000),
         (3, 8200), (2, 16385), (1, 40001), (700, 3000), (1, 16384)]


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantize_is_the_definition(fmt, group, rows, cols):
    torch, q8 = _q8()
    rng = np.random.default_rng(rows * 10007 + cols)
    a = _activations(rng, rows, cols)
    for dtype in (torch.bfloat16, torch.float32):
        _check(q8, torch, torch.from_numpy(a).to(dtype).cuda(), fmt, group)


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
def test_quotients_next_to_every_tie(fmt):
    """Rows whose elements lie on, one step below and one step above every midpoint of codes."""
    torch, q8 = _q8()
    lv = R.levels(fmt)
    mid = (lv[1:] + lv[:-1]) / 2
    rng = np.random.default_rng(5)
    x = []
    for top in np.concatenate([[448.0, 127.0, 1.0, 3.0], np.exp(rng.uniform(-20, 20, 60))]):
        s = np.maximum(np.float32(np.float32(top) / R.TOP[fmt]), np.float32(2.0 ** -100))
        at = (mid * float(s)).astype(np.float32)
        row = np.concatenate([at, np.nextafter(at, np.float32(0)),
                              np.nextafter(at, np.float32(np.inf)), [np.float32(top)]])
        x.append(np.where(np.abs(row) <= top, row, 0))
    x = np.array(x, np.float32) * rng.choice([-1, 1], (len(x), len(x[0]))).astype(np.float32)
    _check(q8, torch, torch.from_numpy(x).cuda(), fmt, 0)


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("group", [0, 128])
def test_extremes(fmt, group):
    """Infinities and NaNs make their row's or group's values NaN and no others; subnormals and
    the largest numbers keep to the definition."""
    torch, q8 = _q8()
    rng = np.random.default_rng(1)
    for cols in (96, 300, 4200):
        x = rng.standard_normal((12, cols)).astype(np.float32)
        x[0, 3], x[1, cols - 1], x[2, 40] = np.inf, np.nan, -np.inf
        x[3] *= np.float32(1e-38)
        x[4] = np.float32(1e-45) * rng.integers(-9, 9, cols)
        x[5] *= np.float32(3e37)
        x[6] = 0
        x[7] = np.where(rng.random(cols) < 0.5, np.float32(3.3e38), np.float32(1.0))
        x[8] = np.finfo(np.float32).max
        x[9] *= np.float32(2.0 ** -100)
        x[10] *= np.float32(2.0 ** -93)
        _check(q8, torch, torch.from_numpy(x).cuda(), fmt, group)


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
def test_every_code_reads_back(fmt):
    torch, q8 = _q8()
    byte = np.tile(np.arange(256, dtype=np.uint8), (3, 1))
    s = np.array([1.0, 0.37, 2.0 ** -100], np.float32)
    t = q8.Q8Tensor(3, 256, fmt, 0, torch.from_numpy(byte).cuda(), torch.from_numpy(s).cuda())
    y = q8.dequantize(t, torch.float32).cpu().numpy()
    want = (R.code_values(byte, fmt) * s[:, None].astype(np.float64)).astype(np.float32)
    np.testing.assert_array_equal(y, want)


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("cols", [100, 200, 513, 2100])
def test_rows_at_every_alignment(fmt, group, cols):
    """Rows inside a wider matrix, of any address and stride, with what lies around them kept."""
    torch, q8 = _q8()
    rng = np.random.default_rng(cols)
    for dtype, off, extra in [(torch.bfloat16, o, e) for o in (0, 1, 3, 8) for e in (0, 5, 16)] + \
                             [(torch.float32, o, e) for o in (0, 1, 2) for e in (3, 8)]:
        ld, rows = cols + extra, 37
        wide = torch.from_numpy(_activations(rng, rows, ld)).to(dtype).cuda()
        flat = torch.empty(off + rows * ld, dtype=dtype, device="cuda")
        x = flat[off:].view(rows, ld)[:, :cols]
        x.copy_(wide[:, :cols])
        t = q8.quantize(x, fmt, group)
        _check(q8, torch, x, fmt, group, t)
        out = torch.full((off + rows * ld + 9,), 77.0, dtype=dtype, device="cuda")
        view = out[off:off + rows * ld].view(rows, ld)[:, :cols]
        assert q8.dequantize(t, out=view) is view
        assert torch.equal(view, q8.dequantize(t, dtype))
        assert (out[:off] == 77).all() and (out[off + rows * ld:] == 77).all()
        if extra:
            assert (out[off:off + rows * ld].view(rows, ld)[:, cols:] == 77).all()


def test_no_rows_leading_dimensions_and_streams():
    torch, q8 = _q8()
    t = q8.quantize(torch.empty(0, 64, device="cuda"), "int8")
    assert q8.dequantize(t).shape == (0, 64)
    x = torch.randn(2, 3, 5, 200, device="cuda")
    t = q8.quantize(x, "e4m3", 128)
    assert (t.rows, t.cols) == (30, 200)
    _check(q8, torch, x, R.E4M3, 128, t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    u = q8.quantize(x, "e4m3", 128, stream=side.cuda_stream)
    y = q8.dequantize(u, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(y, q8.dequantize(t))


def test_offsets_past_32_bits():
    """The last rows of a matrix whose codes and elements lie past 2^31 bytes."""
    torch, q8 = _q8()
    rows, cols = (1 << 21) + 3, 1040
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, cols, device="cuda").bfloat16()
    x[0] = x[-1]
    for group in (0, 128):
        t = q8.quantize(x, "int8", group)
        y = q8.dequantize(t)
        want = q8.dequantize(q8.quantize(x[-3:], "int8", group))
        assert torch.equal(y[-3:], want) and torch.equal(y[0], want[2])
        assert not y[1:-3].any()
        del t, y


# ---- norms --------------------------------------------------------------------


def _norm_case(rows, C, dt, z, fmt, group, pre="rms", w=True, seed=0, **kw):
    """Runs a norm with h in 8 bits beside the same norm with fp32 h (its tests: test_gpu_norm):
    x' is the same, and the codes are those of h, but where 64 bits of h lie within its fp32
    error of a midpoint."""
    torch, q8 = _q8()
    from cnn_convolution_gemm_gb300 import binding as B
    from cnn_convolution_gemm_gb300.norm import ResidualNorm
    rng = np.random.default_rng(rows * 31 + C + seed)
    dtype = getattr(torch, dt)
    x = torch.from_numpy(_activations(rng, rows, C)).to(dtype).cuda()
    zt = torch.from_numpy(_activations(rng, rows, C)).to(dtype).cuda() if z else None
    kind = {"rms": B.CONV_NORM_RMS, "layer": B.CONV_NORM_LAYER}[pre]
    wt = torch.from_numpy((1 + 0.2 * rng.standard_normal(C)).astype(np.float32)).cuda() if w else None
    norm = ResidualNorm(C, dtype, eps=1e-6, pre=kind, w_pre=wt, h_q8=fmt, h_group=group, **kw)
    x_out, h = norm(x, zt)
    _sync(torch)
    plain = ResidualNorm(C, dtype, eps=1e-6, pre=kind, w_pre=wt, **kw)
    x_plain, _ = plain(x, zt)
    assert torch.equal(x_out, x_plain)
    v = x.double().cpu().numpy() + (zt.double().cpu().numpy() if z else 0)
    v = v.astype(np.float32).astype(np.float64)  # x' in fp32, one rounding
    if pre == "layer":
        v = v - v.mean(axis=1, keepdims=True)
    v = v / np.sqrt((v * v).mean(axis=1, keepdims=True) + 1e-6)
    if w:
        v = v * wt.double().cpu().numpy()
    got, pad, s = unpack(h)
    assert not pad.any()
    # fp32 sums of C squares in blocks, root, quotient, weight: within 2^-20 (layer norm: the mean's
    # error, of the row's size, too)
    err = 2.0 ** -20 * (np.abs(v) + (np.abs(v).max(axis=1, keepdims=True) if pre == "layer" else 0))
    # a scale is max |h| / T: off by the largest err of its group / T, and two roundings (a layer
    # norm's err holds the row's largest value, which a group of small ones does not come near)
    want_s = R.scales(v.astype(np.float32), fmt, group)
    room = np.pad(err, ((0, 0), (0, -C % (group or C)))).reshape(rows, -1, group or C).max(axis=2)
    assert (np.abs(s - want_s.astype(np.float64)) <= room / R.TOP[fmt] + 2.0 ** -22 * want_s).all()
    wide = np.repeat(s.astype(np.float64), group or C, axis=1)[:, :C]
    q = v / wide
    unit = np.ones_like(q) if fmt == R.INT8 else \
        2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(q), 1e-9))), -6) - 3)
    # the code is within half a unit of q (the unit of the binade above, next to it)
    room = err / wide + 2.0 ** -18 * np.abs(q)
    assert (np.abs(got - q) <= unit * 0.5 + room).all(), np.max(np.abs(got - q) - unit * 0.5 - room)


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("rows,C", [(1, 32), (1, 4096), (5, 67), (300, 100), (7, 250), (64, 512),
                                    (33, 1001), (9, 1024), (17, 2048), (3, 2579), (40, 4096),
                                    (5, 8192), (3, 8200), (2, 16384), (2, 20000), (1300, 768),
                                    (1300, 2048), (1300, 2560), (1300, 4096), (700, 5120),
                                    (700, 8192), (500, 16384)])
def test_norm(fmt, group, rows, C):
    for dt, z in (("bfloat16", True), ("float32", True), ("bfloat16", False)):
        _norm_case(rows, C, dt, z, fmt, group)


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("rows,C", [(9, 100), (33, 1001), (40, 1024), (1300, 768), (300, 4096),
                                    (5, 8200), (3, 20000)])
def test_fp32_norms_round_step_by_step(fmt, group, rows, C):
    """x and z are whole numbers, so the sum of squares (below 2^24) is exact in any order, and
    every other step is one fp32 operation: codes and scales follow to the bit."""
    torch, q8 = _q8()
    from cnn_convolution_gemm_gb300 import binding as B
    from cnn_convolution_gemm_gb300.norm import ResidualNorm
    rng = np.random.default_rng(rows + C)
    x, z = (rng.integers(-10, 11, (rows, C)).astype(np.float32) for _ in range(2))
    w = (1 + 0.2 * rng.standard_normal(C)).astype(np.float32)
    norm = ResidualNorm(C, torch.float32, eps=1e-6, pre=B.CONV_NORM_RMS,
                        w_pre=torch.from_numpy(w).cuda(), h_q8=fmt, h_group=group)
    _, h = norm(torch.from_numpy(x).cuda(), torch.from_numpy(z).cuda())
    _sync(torch)
    v = x + z
    mean = (v * v).sum(axis=1, keepdims=True, dtype=np.float64).astype(np.float32) * \
        (np.float32(1) / np.float32(C))
    v = v / np.sqrt(mean + np.float32(1e-6)) * w
    assert v.dtype == np.float32
    code, s = R.quantize(v, fmt, group)
    got, pad, got_s = unpack(h)
    np.testing.assert_array_equal(got_s, s)
    np.testing.assert_array_equal(got, code)
    assert not pad.any()


def test_fp32_norms_of_rows_whose_squares_overflow():
    """The root is infinite, the quotients 0; a row with an infinity is NaN, as everywhere."""
    torch, q8 = _q8()
    from cnn_convolution_gemm_gb300 import binding as B
    from cnn_convolution_gemm_gb300.norm import ResidualNorm
    for C in (100, 1001, 4096):
        x = torch.ones(3, C, device="cuda")
        x[0] = 3e19
        x[1, 5] = float("inf")
        _, h = ResidualNorm(C, torch.float32, pre=B.CONV_NORM_RMS, h_q8="int8")(x)
        y = q8.dequantize(h, torch.float32)
        _sync(torch)
        assert not y[0].any() and y[1].isnan().all() and (y[2] - 1).abs().max() < 1e-5


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("group", [0, 128])
def test_layer_norms_and_no_weights(fmt, group):
    _norm_case(70, 640, "bfloat16", True, fmt, group, pre="layer")
    _norm_case(70, 641, "float32", False, fmt, group, pre="layer", w=False)
    _norm_case(1300, 4096, "float32", True, fmt, group, w=False)


def test_norm_types_strides_and_bad_rows():
    """fp32 z into a bf16 stream, rows inside wider matrices, in place; a NaN stays in its row."""
    torch, q8 = _q8()
    from cnn_convolution_gemm_gb300 import binding as B
    from cnn_convolution_gemm_gb300.norm import ResidualNorm
    rng = np.random.default_rng(3)
    for C, rows in ((1000, 40), (512, 2000)):
        x = torch.from_numpy(_activations(rng, rows, C)).bfloat16().cuda()
        z = torch.from_numpy(_activations(rng, rows, C)).cuda()
        z[3, 5], x[7, 9] = float("nan"), float("inf")
        gate = torch.rand(rows, C, device="cuda").bfloat16()
        for group in (0, 128):
            norm = ResidualNorm(C, torch.bfloat16, torch.float32, pre=B.CONV_NORM_RMS,
                                post=B.CONV_NORM_RMS, gate=B.CONV_GATE_SIGMOID, h_q8="e4m3",
                                h_group=group, h_dtype=torch.bfloat16)
            xa, ha = norm(x, z, gate)
            wide = torch.empty(rows, C + 24, device="cuda")
            wide[:, :C] = z
            y = x.clone()
            xb, hb = norm(y, wide[:, :C], gate, x_out=y)
            _sync(torch)
            assert torch.equal(torch.nan_to_num(xa), torch.nan_to_num(xb)) and xb is y
            va, vb = q8.dequantize(ha), q8.dequantize(hb)
            bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
            bad[3] = bad[7] = True
            assert torch.equal(va[~bad], vb[~bad])
            assert torch.isnan(va[3]).all() and not torch.isnan(va[~bad]).any()
            # inf / sqrt(inf) is NaN, what stands beside it 0 / sqrt(inf) = 0: not finite are the
            # row's scale, or its first group's
            assert torch.isnan(va[7, :group or C]).all() and not va[7, group or C:].any()


def test_norm_into_its_buffers_and_graphs():
    torch, q8 = _q8()
    from cnn_convolution_gemm_gb300 import binding as B
    from cnn_convolution_gemm_gb300.norm import ResidualNorm
    norm = ResidualNorm(768, pre=B.CONV_NORM_RMS, h_q8="int8", h_group=128)
    x = torch.randn(50, 768, device="cuda").bfloat16()
    h = q8.empty(50, 768, "int8", "cuda", 128)
    assert norm(x, h_out=h)[1] is h
    with pytest.raises(ValueError):
        norm(x, h_out=q8.empty(50, 768, "int8", "cuda", 0))
    with pytest.raises(ValueError):
        norm(x[:49], h_out=h)
    y = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm(x, h_out=h)
        q8.dequantize(h, out=y)
        again = q8.quantize(y, "e4m3")
    for seed in range(3):
        torch.manual_seed(seed)
        x.copy_(torch.randn(50, 768, device="cuda"))
        graph.replay()
        want = q8.dequantize(norm(x)[1])
        assert torch.equal(y, want)
        assert torch.equal(q8.dequantize(again), q8.dequantize(q8.quantize(want, "e4m3")))
