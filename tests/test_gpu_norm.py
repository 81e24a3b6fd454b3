"""The norms around a residual block against 64 bits, and the 4-bit residual block."""
import numpy as np
import pytest

from tests import fp4_ref as R
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu
B = R.B
EPS = 1e-6


def _norm():
    torch = need_gpu()
    from cnn_convolution_gemm_gb300.norm import ResidualNorm
    return torch, ResidualNorm


def _case(post, pre, rows, C, gate=0, gate_rows=1, dt="bfloat16", zdt=None, h_fmt=None, rs=0.5,
          offset=0.0, weights=True, strided=False, with_z=True, in_place=False):
    """Runs one case and compares it with 64 bits.  Tolerance: a row's sums are added in fp32
    in at most C / 32 + 10 dependent steps (relative 2^-24 each, halved on average by nothing:
    taken in full), the rest of a value is a dozen fp32 operations; layer norms subtract the
    mean, so the error is relative to the largest magnitude before the subtraction."""
    torch, ResidualNorm = _norm()
    rng = np.random.default_rng(rows * 31 + C * 7 + post + 3 * pre + 11 * gate)
    zdt = zdt or dt
    xd, zd = getattr(torch, dt), getattr(torch, zdt)
    up = lambda a, d: torch.from_numpy(np.ascontiguousarray(a)).to(d).cuda()  # noqa: E731
    size = np.exp(0.5 * rng.standard_normal(C))
    x = up(rng.standard_normal((rows, C)) * size * 4 + offset, xd)
    z = up(rng.standard_normal((rows, C)) * size + offset, zd) if with_z else None
    g = up(rng.standard_normal((-(-rows // gate_rows), C)), zd) if gate and with_z else None
    if strided:
        x = torch.cat([x, x[:, :1]], 1)[:, :C]
        z = torch.cat([z, z[:, :1], z[:, :1]], 1)[:, :C]
    vec = lambda s, o: up(o + s * rng.standard_normal(C), torch.float32)  # noqa: E731
    p = {"w_post": vec(0.1, 1) if weights and post else None,
         "b_post": vec(0.1, 0) if weights and post == B.CONV_NORM_LAYER else None,
         "w_pre": vec(0.1, 1) if weights and pre else None,
         "b_pre": vec(0.1, 0) if weights and pre == B.CONV_NORM_LAYER else None}
    h_scale = 1.0 if h_fmt != R.NV else float(np.float32(0.0041))
    layer = ResidualNorm(C, xd, zd, eps=EPS, post=post, pre=pre, gate=gate, gate_rows=gate_rows,
                         residual_scale=rs, h_fmt=h_fmt, h_scale=h_scale, **p)
    x64 = x.double().cpu().numpy()
    x_out = x if in_place else None
    if strided:
        big = torch.full((rows, C + 9), 7.0, dtype=xd, device="cuda")
        x_out = big[:, 4:4 + C]
    xo, h = layer(x, z, gate=g, x_out=x_out)
    B.conv_sync_status(torch.cuda.current_stream().cuda_stream)
    n64 = {k: None if v is None else v.double().cpu().numpy() for k, v in p.items()}
    steps = (C / 32 + 10 + 12) * 2.0 ** -24
    want, bound = x64, 4 * 2.0 ** -24 * np.abs(x64)
    if with_z:
        z64 = z.double().cpu().numpy()
        u = R.norm(z64, post, EPS, n64["w_post"], n64["b_post"])
        gg = np.float64(rs)
        if gate:
            gv = g.double().cpu().numpy()
            gv = 1 / (1 + np.exp(-gv)) if gate == B.CONV_GATE_SIGMOID else gv
            gg = rs * gv[np.arange(rows) // gate_rows]
        rstd = _rstd(z64, post)
        amp = np.abs(z64) * rstd if post != B.CONV_NORM_LAYER else (
            (np.abs(z64) + np.abs(z64).max(axis=1, keepdims=True)) * rstd)
        w = 1 if n64["w_post"] is None else np.abs(n64["w_post"])
        ub = steps * (amp * w + (0 if n64["b_post"] is None else np.abs(n64["b_post"])))
        want = x64 + gg * u
        bound = bound + np.abs(gg) * (ub + 8 * 2.0 ** -24 * np.abs(u)) + 4 * 2.0 ** -24 * np.abs(want)
    ulp = {"bfloat16": 2.0 ** -8, "float32": 2.0 ** -24}
    off = np.abs(xo.double().cpu().numpy() - want)
    assert (off <= bound + ulp[dt] * np.abs(want) + 1e-37).all(), (off / (bound + ulp[dt] * np.abs(want))).max()
    if strided:
        assert (big[:, :4] == 7).all() and (big[:, 4 + C:] == 7).all()
    if not pre:
        assert h is None
        return
    wanth = R.norm(want, pre, EPS, n64["w_pre"], n64["b_pre"])
    rstd = _rstd(want, pre)
    amp = np.abs(want) + (np.abs(want).max(axis=1, keepdims=True) if pre == B.CONV_NORM_LAYER else 0)
    w = 1 if n64["w_pre"] is None else np.abs(n64["w_pre"])
    # the error of x' enters directly and through the row's statistics
    through = bound + np.sqrt((bound ** 2).mean(axis=1, keepdims=True)) * (
        1 + np.abs(want) * rstd * (2 if pre == B.CONV_NORM_LAYER else 1))
    hb = (steps * amp + through) * rstd * w + steps * (0 if n64["b_pre"] is None else np.abs(n64["b_pre"]))
    if h_fmt is not None:
        R.check_quantized(h, wanth, hb, h_fmt, h_scale)
        return
    off = np.abs(h.double().cpu().numpy() - wanth)
    assert (off <= hb + ulp[zdt] * np.abs(wanth) + 1e-37).all(), (off / (hb + ulp[zdt] * np.abs(wanth))).max()


def _rstd(v, kind):
    if kind == B.CONV_NORM_NONE:
        return 1.0
    m = v.mean(axis=1, keepdims=True) if kind == B.CONV_NORM_LAYER else 0.0
    return 1 / np.sqrt(((v - m) ** 2).mean(axis=1, keepdims=True) + EPS)


N, RMS, LN = B.CONV_NORM_NONE, B.CONV_NORM_RMS, B.CONV_NORM_LAYER


@pytest.mark.parametrize("rows,C", [(1, 1), (1, 4096), (3, 7), (5, 32), (130, 64), (9, 100), (33, 257),
                                    (17, 1000), (4, 1001), (300, 768), (7, 2048), (5, 4100), (3, 8192),
                                    (2, 12345), (2, 16384), (2, 32768)])
@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_rms_both_sides(rows, C, dt):
    _case(RMS, RMS, rows, C, dt=dt)


@pytest.mark.parametrize("post,pre", [(N, RMS), (RMS, N), (N, LN), (LN, LN), (LN, RMS), (RMS, LN), (N, N)])
@pytest.mark.parametrize("rows,C", [(5, 96), (33, 515), (6, 2304)])
def test_norm_kinds(post, pre, rows, C):
    _case(post, pre, rows, C)
    _case(post, pre, rows, C, dt="float32", weights=False)


@pytest.mark.parametrize("gate", [B.CONV_GATE_LINEAR, B.CONV_GATE_SIGMOID])
@pytest.mark.parametrize("rows,C,gate_rows", [(6, 128, 1), (50, 200, 7), (49, 256, 49), (10, 96, 1000)])
def test_gates(gate, rows, C, gate_rows):
    _case(RMS, RMS, rows, C, gate, gate_rows)
    _case(LN, LN, rows, C, gate, gate_rows, dt="float32", zdt="bfloat16")


@pytest.mark.parametrize("h_fmt", [R.MX, R.NV])
@pytest.mark.parametrize("rows,C", [(1, 2048), (3, 40), (130, 288), (7, 1000), (2, 4096), (140, 64)])
def test_quantized_output(h_fmt, rows, C):
    _case(RMS, RMS, rows, C, h_fmt=h_fmt)
    _case(LN, LN, rows, C, dt="float32", zdt="bfloat16", h_fmt=h_fmt, gate=2)


@pytest.mark.parametrize("post,pre,rows,C,kw", [
    (RMS, RMS, 1301, 8192, {}), (LN, LN, 1301, 8192, {}), (LN, LN, 1300, 8192, {"dt": "float32"}),
    (RMS, LN, 2501, 4096, {"gate": 2, "gate_rows": 7}), (LN, RMS, 2501, 4096, {"dt": "float32"}),
    (N, RMS, 10001, 1024, {}), (RMS, N, 10001, 1024, {"gate": 1, "gate_rows": 196}),
    (RMS, RMS, 5003, 2048, {"h_fmt": R.MX}), (LN, LN, 5003, 2040, {"h_fmt": R.NV, "gate": 1}),
    (RMS, RMS, 1303, 7000, {"in_place": True}), (RMS, RMS, 2501, 4096, {"dt": "float32", "zdt": "bfloat16"}),
    (RMS, RMS, 701, 12296, {}), (LN, LN, 611, 16384, {"gate": 1}), (LN, LN, 500, 9000, {"dt": "float32", "h_fmt": R.NV}),
    (N, LN, 600, 16376, {"with_z": False, "h_fmt": R.MX}), (LN, LN, 520, 4104, {"gate": 2, "gate_rows": 3}),
    (RMS, RMS, 1303, 8192, {"weights": False}), (RMS, RMS, 3001, 4001, {}), (N, LN, 3001, 4096, {"with_z": False})])
def test_many_rows(post, pre, rows, C, kw):
    """Rows that come ahead of their turn, two at a time, and an odd one last."""
    _case(post, pre, rows, C, **kw)


@pytest.mark.parametrize("rows,C", [(1, 16), (3, 128), (1037, 48), (20003, 112), (5, 144), (2051, 256), (1037, 90), (517, 250)])
@pytest.mark.parametrize("kw", [{}, {"dt": "float32", "gate": 2, "gate_rows": 5}, {"h_fmt": R.MX, "gate": 1},
                                {"h_fmt": R.NV, "dt": "float32", "zdt": "bfloat16"}, {"in_place": True}], ids=str)
def test_narrow_rows_share_warps(rows, C, kw):
    _case(LN, RMS, rows, C, **kw)


def test_mixed_types_strides_in_place_and_first_norm():
    _case(RMS, LN, 20, 320, dt="float32", zdt="bfloat16")
    _case(RMS, LN, 20, 320, dt="bfloat16", zdt="float32")
    for C in (95, 256):
        _case(RMS, RMS, 12, C, strided=True)
        _case(LN, RMS, 12, C, strided=True, dt="float32")
        _case(RMS, RMS, 40, C, in_place=True)
        _case(N, RMS, 12, C, with_z=False)
        _case(N, LN, 12, C, with_z=False, h_fmt=R.MX)


def test_large_means_keep_their_digits():
    """Layer norms of rows whose mean is a thousand times their deviation."""
    _case(LN, LN, 9, 1024, dt="float32", offset=4000.0)
    _case(LN, LN, 9, 300, dt="float32", offset=-4000.0)


def test_zero_rows_and_rows_of_zeros():
    torch, ResidualNorm = _norm()
    layer = ResidualNorm(64, post=RMS, pre=RMS)
    n = B.conv_launch_count()
    x, h = layer(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"),
                 torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))
    assert x.shape == h.shape == (0, 64) and B.conv_launch_count() == n
    z = torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda")
    x, h = layer(z, z)
    assert not x.any() and not h.any()
    # an infinity or a NaN stays in its row
    z[1, 5] = float("inf")
    x, h = layer(torch.ones_like(z), z)
    assert torch.isnan(x[1, 5]) and torch.isnan(h[1]).all()
    assert torch.isfinite(x[[0, 2]]).all() and torch.isfinite(h[[0, 2]]).all()


def test_other_stream_and_determinism():
    torch, ResidualNorm = _norm()
    layer = ResidualNorm(1000, post=LN, pre=RMS)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, z = (torch.randn(700, 1000, generator=gen, device="cuda").bfloat16() for _ in range(2))
    want = layer(x, z)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(5):
        got = layer(x, z, stream=s.cuda_stream)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("fmt", [R.MX, R.NV])
@pytest.mark.parametrize("rows,C,hidden", [(1, 256, 512), (70, 96, 200), (300, 256, 640)])
def test_residual_block(fmt, rows, C, hidden):
    """Two chained blocks against 64 bits.  A 4-bit value within the fp32 error of a rounding
    boundary may go either way, which moves a product by a few times 2^-5 of one term:
    the comparison is over the norm of the difference."""
    torch = need_gpu()
    from cnn_convolution_gemm_gb300.residual_block import Fp4ResidualBlock
    rng = np.random.default_rng(rows + C)
    up = lambda a, d=torch.float32: torch.from_numpy(np.ascontiguousarray(a)).to(d).cuda()  # noqa: E731
    g = 1.0 if fmt == R.MX else float(np.float32(0.0052))
    gw = 1.0 if fmt == R.MX else float(np.float32(0.00037))
    x = up(3 * rng.standard_normal((rows, C)), torch.bfloat16)
    gate = up(rng.standard_normal((1, C)), torch.bfloat16)
    norms = [1 + 0.1 * rng.standard_normal(C) for _ in range(5)]
    nt = [up(n) for n in norms]
    blocks, weights = [], []
    for i in range(2):
        w1, w2 = rng.standard_normal((hidden, C)) / np.sqrt(C), rng.standard_normal((C, hidden)) / np.sqrt(hidden)
        b1, b2 = 0.1 * rng.standard_normal(hidden), 0.1 * rng.standard_normal(C)
        blk = Fp4ResidualBlock(C, hidden, fmt, residual_scale=0.5, gate=B.CONV_GATE_LINEAR, gate_rows=rows,
                               w_pre=nt[2 * i], w_post=nt[2 * i + 1], w_next=nt[2 * i + 2], b1=up(b1), b2=up(b2),
                               h_scale=g, t_scale=g, chain=i == 0, next_scale=g)
        blk.prepack(up(w1, torch.bfloat16), up(w2, torch.bfloat16), gw, gw)
        blocks.append(blk)
        weights.append((R.tensor_values(blk.fc1.w), R.tensor_values(blk.fc2.w),
                        blk.b1.double().cpu().numpy(), blk.b2.double().cpu().numpy()))
    xo, h = blocks[0](x, gate=gate)
    assert h.rows == rows and h.fmt == fmt
    xo, h = blocks[1](xo, gate=gate, h=h)
    B.conv_sync_status(torch.cuda.current_stream().cuda_stream)
    v = x.double().cpu().numpy()
    n64 = [n.double().cpu().numpy() for n in nt]
    q = lambda a: R.values(*R.quantize(a.astype(np.float32), fmt, g), fmt, a.shape[1], g)  # noqa: E731
    for i, (w1, w2, b1, b2) in enumerate(weights):
        t = R.activate(q(R.norm(v, RMS, EPS, n64[2 * i])) @ w1.T + b1, B.CONV_ACT_GELU)
        zz = q(t) @ w2.T + b2
        v = v + 0.5 * gate.double().cpu().numpy() * R.norm(zz, RMS, EPS, n64[2 * i + 1])
        hh = R.norm(v, RMS, EPS, n64[2 * i + 2])
    for got, want in ((xo, v), (h, hh)):
        off = np.linalg.norm(got.double().cpu().numpy() - want) / np.linalg.norm(want)
        assert off <= 0.01, off


def test_residual_block_is_its_parts():
    """The block's one call against the layers called one by one: bit for bit; strided x and
    outputs, x' in place, another stream, weights exchanged in a layer of the block."""
    torch = need_gpu()
    from cnn_convolution_gemm_gb300.residual_block import Fp4ResidualBlock
    torch.manual_seed(3)
    rows, C, hidden = 37, 160, 352
    w = [1 + 0.1 * torch.randn(C, device="cuda") for _ in range(3)]
    blk = Fp4ResidualBlock(C, hidden, B.CONV_FP4_MX, residual_scale=0.5, gate=B.CONV_GATE_SIGMOID, gate_rows=10,
                           w_pre=w[0], w_post=w[1], w_next=w[2], b1=torch.randn(hidden, device="cuda"))
    rand = lambda *s: torch.randn(*s, device="cuda").bfloat16()  # noqa: E731
    blk.prepack(rand(hidden, C), rand(C, hidden))
    gate = rand(4, C)

    def parts(x, x_out=None):
        h = blk.norm_in(x, want_x=False)[1]
        z = blk.fc2(blk.fc1(h, bias=blk.b1))
        return blk.norm_out(x, z, gate=gate, x_out=x_out)

    def same(got, want):
        return all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(got, want))
    x = rand(rows, C)
    want = [t.clone() for t in parts(x)]
    assert same(blk(x, gate=gate), want)
    wide, out = rand(rows, C + 9), torch.empty(rows, C + 5, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:3 + C] = x
    at, to = wide[:, 3:3 + C], out[:, 2:2 + C]
    strided = [t.clone() for t in parts(at, to)]
    to.zero_()
    assert same([t.contiguous() for t in blk(at, gate=gate, x_out=to)], strided)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = x.clone()
        got = blk(y, gate=gate, x_out=y)
    s.synchronize()
    assert got[0] is y and same(got, want)
    blk.fc1.prepack(rand(hidden, C))
    want = [t.clone() for t in parts(x)]
    assert same(blk(x, gate=gate), want)
    B.conv_sync_status(torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("fmt", [B.CONV_FP4_MX, B.CONV_FP4_NV])
@pytest.mark.parametrize("rows", [2, 2600])
def test_residual_block_workspace_at_16_bytes(fmt, rows):
    """A workspace that lies on 16 bytes and not on 32 holds the same bits of h, t and z.  The
    norm behind takes z's rows by single columns then, and adds their squares in another order
    (2^-20 of |x| + |u| < 32): x' and h' may round to the next bf16 value."""
    torch = need_gpu()
    from cnn_convolution_gemm_gb300.residual_block import Fp4ResidualBlock
    torch.manual_seed(5)
    C, hidden = 256, 2112
    blk = Fp4ResidualBlock(C, hidden, fmt)
    blk.prepack(torch.randn(hidden, C, device="cuda"), torch.randn(C, hidden, device="cuda"))
    x = torch.randn(rows, C, device="cuda").bfloat16()
    blk(x)  # gives the descriptor its weights
    need = B.conv_fp4_block_workspace_size(blk.desc, rows)
    stream = torch.cuda.current_stream().cuda_stream
    runs = []
    for off in (0, 16):
        buf = torch.zeros(need + 64, dtype=torch.uint8, device="cuda")
        at = off + -buf.data_ptr() % 32
        out = [torch.empty_like(x) for _ in range(2)]
        B.conv_fp4_block_fwd(blk.desc, rows, x.data_ptr(), None, None, None, out[0].data_ptr(),
                             out[1].data_ptr(), None, buf.data_ptr() + at, need, stream)
        B.conv_sync_status(stream)
        assert not buf[:at].any() and not buf[at + need:].any()
        runs.append((buf[at:at + need], out))
    assert torch.equal(runs[0][0], runs[1][0])
    for a, b in zip(runs[0][1], runs[1][1]):
        a, b = a.float(), b.float()
        assert ((a - b).abs() <= 2.0 ** -7 * torch.maximum(a.abs(), b.abs()) + 2.0 ** -15).all()


def test_residual_block_after_strided_calls_of_its_parts():
    """Parts called with strided tensors leave the block's own calls as they were."""
    torch = need_gpu()
    from cnn_convolution_gemm_gb300.residual_block import Fp4ResidualBlock
    torch.manual_seed(6)
    rows, C, hidden = 20, 96, 160
    blk = Fp4ResidualBlock(C, hidden, B.CONV_FP4_MX, gate=B.CONV_GATE_LINEAR)
    rand = lambda *s: torch.randn(*s, device="cuda").bfloat16()  # noqa: E731
    blk.prepack(rand(hidden, C), rand(C, hidden))
    x, gate = rand(rows, C), rand(rows, C)
    want = [t.clone() for t in blk(x, gate=gate)]
    at = lambda t: torch.cat([t, t], 1)[:, :C]  # noqa: E731
    h = blk.norm_in(at(x), x_out=at(x))[1]
    z = blk.fc2(blk.fc1(h), out=torch.zeros(rows, 2 * C, dtype=blk.fc2.y_dtype, device="cuda")[:, :C])
    blk.norm_out(at(x), z, gate=at(gate), x_out=at(x), h_out=at(x))
    got = blk(x, gate=gate)
    B.conv_sync_status(torch.cuda.current_stream().cuda_stream)
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(got, want))


def _block_behind_its_codes(dt, fmt, rows, C, hidden, gate_rows, strided=False):
    """x' and h' of a block against 64 bits over the 4-bit t that its own first layer gives, so
    that no code can fall to another side: z within the product's bound, whose share reaches u
    directly and through the row's norm (relative rstd * rms(error)); sums of at most C / 32 + 22
    steps of 2^-24 as in _case; one rounding to dt at the end."""
    torch = need_gpu()
    from cnn_convolution_gemm_gb300.residual_block import Fp4ResidualBlock
    rng = np.random.default_rng(rows + C)
    dtype = getattr(torch, dt)
    up = lambda a, d=torch.float32: torch.from_numpy(np.ascontiguousarray(a)).to(d).cuda()  # noqa: E731
    n64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    g = 1.0 if fmt == R.MX else float(np.float32(0.0052))
    gw = 1.0 if fmt == R.MX else float(np.float32(0.00037))
    x = up(0.05 * rng.standard_normal((rows, C)), dtype)
    gate = up(rng.standard_normal((-(-rows // gate_rows), C)), dtype)
    w = [up(1 + 0.1 * rng.standard_normal(C)) for _ in range(3)]
    b1, b2 = up(0.1 * rng.standard_normal(hidden)), up(0.1 * rng.standard_normal(C))
    blk = Fp4ResidualBlock(C, hidden, fmt, dtype, residual_scale=0.5, gate=B.CONV_GATE_LINEAR,
                           gate_rows=gate_rows, w_pre=w[0], w_post=w[1], w_next=w[2], b1=b1, b2=b2,
                           h_scale=g, t_scale=g)
    blk.prepack(up(rng.standard_normal((hidden, C)) / np.sqrt(C)),
                up(rng.standard_normal((C, hidden)) / np.sqrt(hidden)), gw, gw)
    if strided:
        x = torch.cat([x, x[:, :3]], 1)[:, :C]
    xo, h = blk(x, gate=gate)
    t = blk.fc1(blk.norm_in(x, want_x=False)[1], bias=b1)
    B.conv_sync_status(torch.cuda.current_stream().cuda_stream)
    assert xo.dtype is dtype and h.dtype is dtype
    tv, wv = R.tensor_values(t), R.tensor_values(blk.fc2.w)
    z = tv @ wv.T + n64(b2)
    z_err = R.product_bound(tv, wv, z, np.abs(n64(b2)), 24)
    steps = (C / 32 + 22) * 2.0 ** -24
    rms = lambda v: np.sqrt((v ** 2).mean(axis=1, keepdims=True))  # noqa: E731

    def normed(v, err, weight):
        rstd = _rstd(v, RMS)
        n = v * rstd * weight
        return n, np.abs(weight) * rstd * (err + np.abs(v) * rstd * rms(err)) + steps * np.abs(n)
    u, u_err = normed(z, z_err, n64(w[1]))
    gg = 0.5 * n64(gate)[np.arange(rows) // gate_rows]
    want = n64(x) + gg * u
    err = np.abs(gg) * (u_err + 8 * 2.0 ** -24 * np.abs(u)) + 4 * 2.0 ** -24 * (
        np.abs(n64(x)) + np.abs(want))
    want_h, h_err = normed(want, err, n64(w[2]))
    for got, v, e in ((xo, want, err), (h, want_h, h_err)):
        off = np.abs(n64(got) - v)
        assert (off <= e + R.half_spacing(np.abs(v) + e, dt)).all()


@pytest.mark.parametrize("fmt", [R.MX, R.NV])
@pytest.mark.parametrize("rows,C,hidden,gate_rows,strided", [(1, 256, 512, 1, False), (70, 96, 200, 7, False),
                                                             (300, 250, 640, 300, True), (2000, 1024, 512, 1, False)])
def test_residual_block_of_an_fp32_stream(fmt, rows, C, hidden, gate_rows, strided):
    """The stream, the gates and h' in fp32, and nothing between them in fewer bits but h and t."""
    _block_behind_its_codes("float32", fmt, rows, C, hidden, gate_rows, strided)


@pytest.mark.parametrize("fmt", [R.MX, R.NV])
@pytest.mark.parametrize("rows,C,hidden,gate_rows,strided", [(1, 256, 512, 1, False), (70, 96, 200, 7, False),
                                                             (300, 250, 640, 300, True), (2000, 1024, 512, 1, False)])
def test_residual_block_holds_z_in_32_bits(fmt, rows, C, hidden, gate_rows, strided):
    """x' and h' of a bf16 stream are rounded once, at the end."""
    _block_behind_its_codes("bfloat16", fmt, rows, C, hidden, gate_rows, strided)


@pytest.mark.parametrize("post,pre,rows,C,kw", [
    (RMS, RMS, 1, 4096, {"gate": 2}), (LN, LN, 33, 257, {"gate": 1}), (RMS, LN, 5, 96, {}), (N, N, 9, 100, {}),
    (RMS, RMS, 1301, 8192, {}), (LN, LN, 2501, 4096, {"gate": 2, "gate_rows": 7}), (LN, RMS, 10001, 1024, {}),
    (RMS, RMS, 5003, 2040, {"h_fmt": R.NV, "gate": 1}), (RMS, RMS, 1303, 6000, {"in_place": True}),
    (LN, RMS, 701, 12296, {}), (RMS, N, 3, 20000, {}), (RMS, RMS, 4, 9001, {"h_fmt": R.MX}),
    (RMS, LN, 12, 256, {"strided": True}), (LN, RMS, 1037, 112, {"h_fmt": R.MX}), (RMS, RMS, 40, 2500, {}),
    (LN, RMS, 12, 256, {"with_z": False}), (LN, RMS, 12, 95, {"with_z": False, "h_fmt": R.NV})])
def test_z_in_another_type(post, pre, rows, C, kw):
    """fp32 z with bf16 x, gate and h, against the layer that has gate and h in fp32 too (and its
    own test against 64 bits).  Sums may be added in another order: (C / 32 + 22) steps of 2^-24
    of a row's largest magnitude, up to 4 (largest u or h + 1) with the weights and biases here.
    x' differs by 0.5 |g| of that (|g| <= 5, |u| <= 8: 90 steps), then may be the next bf16 value
    (2^-7); h by its own sums, by that of x' (whose deviation is 4: less than half) and by its
    rounding."""
    torch, ResidualNorm = _norm()
    kw = dict(kw)
    gate, gate_rows, h_fmt = kw.pop("gate", 0), kw.pop("gate_rows", 1), kw.pop("h_fmt", None)
    with_z, strided, in_place = (kw.pop(k, d) for k, d in (("with_z", True), ("strided", False),
                                                           ("in_place", False)))
    assert not kw
    gen = torch.Generator(device="cuda").manual_seed(rows + C)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, z = (4 * rand(rows, C)).bfloat16(), rand(rows, C) if with_z else None
    g = rand(-(-rows // gate_rows), C).bfloat16() if gate and with_z else None
    if strided:
        x, z = torch.cat([x, x], 1)[:, :C], torch.cat([z, z[:, :1]], 1)[:, :C]
    vec = lambda o, there: o + 0.1 * rand(C) if there else None  # noqa: E731
    scale = 1.0 if h_fmt != R.NV else float(np.float32(0.0041))
    p = dict(post=post, pre=pre, gate=gate, gate_rows=gate_rows, residual_scale=0.5,
             w_post=vec(1, post), b_post=vec(0, post == LN), w_pre=vec(1, pre), b_pre=vec(0, pre == LN))
    want_x, want_h = ResidualNorm(C, torch.bfloat16, torch.float32, **p)(
        x, z, gate=None if g is None else g.float())
    layer = ResidualNorm(C, torch.bfloat16, torch.float32, h_dtype=torch.bfloat16, h_fmt=h_fmt,
                         h_scale=scale, **p)
    xo, h = layer(x, z, gate=g, x_out=x if in_place else None)
    B.conv_sync_status(torch.cuda.current_stream().cuda_stream)
    a, b = xo.float(), want_x.float()
    steps = (C / 32 + 22) * 2.0 ** -24
    assert ((a - b).abs() <= 2.0 ** -7 * torch.maximum(a.abs(), b.abs()) + 90 * steps).all()
    if not pre:
        assert h is None
        return
    want = want_h.double().cpu().numpy()
    err = steps * (4 * (np.abs(want).max(axis=1, keepdims=True) + 1) + 45) + 0 * want
    if h_fmt is not None:
        R.check_quantized(h, want, err, h_fmt, scale)
        return
    assert h.dtype is torch.bfloat16
    off = np.abs(h.double().cpu().numpy() - want)
    assert (off <= err + R.half_spacing(np.abs(want) + err, "bfloat16")).all()


@pytest.mark.parametrize("dt,zdt,hdt", [("float32", "float32", None), ("float32", "bfloat16", None),
                                        ("bfloat16", "float32", None), ("bfloat16", "bfloat16", None),
                                        ("bfloat16", "float32", "bfloat16")])
@pytest.mark.parametrize("C", [96, 257, 1024])
def test_sigmoid_gates_keep_their_digits(dt, zdt, hdt, C):
    """Gates down to -80, where the sigmoid is exp(-80), against u so large that x' shows them:
    x' = u * sigmoid.  In units of 2^-23: exp 2 (its argument's rounding 0.75 |x| where every
    output has 16 bits), 1 + exp 0.5, the reciprocal 1, products 1.5; then one rounding."""
    torch, ResidualNorm = _norm()
    gd = getattr(torch, hdt or zdt)
    gate = torch.linspace(-80, 20, 5 * C).view(5, C).to(gd).cuda()
    z = torch.full((5, C), 2.0 ** 60, device="cuda").to(getattr(torch, zdt))
    x = torch.zeros(5, C, device="cuda").to(getattr(torch, dt))
    xo, _ = ResidualNorm(C, x.dtype, z.dtype, gate=B.CONV_GATE_SIGMOID, h_dtype=gd)(x, z, gate=gate)
    B.conv_sync_status(torch.cuda.current_stream().cuda_stream)
    g = gate.double().cpu().numpy()
    want = 2.0 ** 60 / (1 + np.exp(-g))
    exact = dt == "float32" or (hdt or zdt) == "float32"
    err = want * (5 + (0 if exact else 0.75 * np.abs(g))) * 2.0 ** -23
    assert (np.abs(xo.double().cpu().numpy() - want) <= err + R.half_spacing(want + err, dt)).all()


@pytest.mark.parametrize("h_fmt", [R.MX, R.NV])
@pytest.mark.parametrize("rows,C", [(1, 9001), (3, 16383), (2, 20001), (2, 32767), (400, 9999)])
def test_quantized_output_of_wide_odd_rows(h_fmt, rows, C):
    """Rows above 8192 channels at addresses that allow no vector accesses, into 4 bits."""
    _case(RMS, RMS, rows, C, h_fmt=h_fmt)
    _case(LN, LN, rows, C, dt="float32", zdt="bfloat16", h_fmt=h_fmt, gate=2)
    _case(N, LN, rows, C, dt="float32", h_fmt=h_fmt, with_z=False)


def test_threads_share_layers_and_blocks():
    """Two threads on one stream, whose tensors have other row strides and numbers of rows: every
    result is the one that a single thread gets, bit for bit.  And blocks of no rows."""
    import threading
    torch = need_gpu()
    from cnn_convolution_gemm_gb300 import fp4
    from cnn_convolution_gemm_gb300.norm import ResidualNorm
    from cnn_convolution_gemm_gb300.residual_block import Fp4ResidualBlock
    torch.manual_seed(7)
    C, K = 160, 288
    rand = lambda *s: torch.randn(*s, device="cuda").bfloat16()  # noqa: E731
    layer, norm, blk = fp4.Fp4Linear(C, K, R.NV, x_scale=0.004), ResidualNorm(C, pre=LN), Fp4ResidualBlock(C, K)
    layer.prepack(rand(K, C), 0.01)
    blk.prepack(rand(K, C), rand(C, K))
    xs = [rand(40, C), rand(75, C + 24)[:, 8:8 + C]]
    calls = [layer, lambda x: norm(x)[1], lambda x: blk(x)[1], lambda x: blk.norm_in(x)[1].codes]
    want = [[f(x).clone() for f in calls] for x in xs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        for _ in range(100):
            for f, w in zip(calls, want[i]):
                if not torch.equal(f(xs[i]), w):
                    wrong.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    B.conv_sync_status(torch.cuda.current_stream().cuda_stream)
    assert not wrong
    x, h = blk(xs[0][:0])
    assert x.shape == h.shape == (0, C)
