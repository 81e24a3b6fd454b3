"""Layers with integer 4-bit weights against 64 bits, on the GPU."""
import numpy as np
import pytest

from tests import w4_ref as R
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu
BF16, F32, E4M3, INT8 = "bf16", "f32", "e4m3", "int8"


def _mods():
    torch = need_gpu()
    from cnn_convolution_gemm_gb300 import binding as B
    from cnn_convolution_gemm_gb300 import q8
    from cnn_convolution_gemm_gb300.w4 import W4Linear
    return torch, B, q8, W4Linear


def _sync(torch, B):
    B.conv_sync_status(torch.cuda.current_stream().cuda_stream)


class Case:
    """A layer with its weights, and their values in 64 bits."""

    def __init__(self, C, K, group=128, x=BF16, y=BF16, zeros=True, scale=BF16, act=0, bias=True,
                 residual=False, x_group=0, seed=0):
        self.torch, self.B, self.q8, W4Linear = _mods()
        torch = self.torch
        self.rng = rng = np.random.default_rng(seed + C * 7 + K)
        self.C, self.K, self.x, self.y, self.act, self.x_group = C, K, x, y, act, x_group
        self.y_dtype = torch.bfloat16 if y == BF16 else torch.float32
        groups = -(-C // group) if group else 1
        q = rng.integers(0, 16, (K, C))
        s = torch.from_numpy((rng.uniform(0.2, 1, (K, groups)) / np.sqrt(C)).astype(np.float32))
        s = s.to(torch.bfloat16 if scale == BF16 else torch.float32)
        z = rng.integers(0, 16, (K, groups)).astype(np.uint8) if zeros else None
        self.w = R.weights(q, s.double().numpy(), z, group)
        self.codes = torch.from_numpy(R.pack_weights(q)).cuda()
        self.scales, self.zeros = s.cuda(), None if z is None else torch.from_numpy(z).cuda()
        more = dict(x_dtype=None, x_q8=x, x_group=x_group) if x in (E4M3, INT8) else \
            dict(x_dtype=torch.bfloat16 if x == BF16 else torch.float32)
        self.layer = W4Linear(C, K, group, y_dtype=self.y_dtype, act=act, has_residual=residual,
                              scale_dtype=s.dtype, **more)
        self.layer.load(self.codes, self.scales, self.zeros)
        self.bias = torch.from_numpy(rng.standard_normal(K).astype(np.float32)).cuda() if bias else None
        self.residual = residual

    def input(self, M):
        """(x, its values in 64 bits)."""
        torch = self.torch
        a = (self.rng.standard_normal((M, self.C)) *
             np.exp(0.5 * self.rng.standard_normal(self.C))).astype(np.float32)
        t = torch.from_numpy(a).cuda()
        if self.x == BF16:
            t = t.bfloat16()
            return t, t.double().cpu().numpy()
        if self.x == F32:
            return t, a.astype(np.float64)
        t = self.q8.quantize(t, self.x, self.x_group)
        code, s = R.quantize(a, {E4M3: R.E4M3, INT8: R.INT8}[self.x], self.x_group)
        return t, R.values(code, s, self.x_group)

    def res(self, M):
        if not self.residual:
            return None
        return self.torch.from_numpy(self.rng.standard_normal((M, self.K)).astype(np.float32)).to(
            self.y_dtype).cuda()

    def expect(self, v, res):
        """(y in 64 bits, how far a call may be off).

        Sums: products are exact; an fp32 sum of C of them, however ordered (the tensor core adds
        at least eight at a time, and truncates: 2^-23 a step), of a group's sums, of the ranges of
        a split reduction, and the roundings of scale * sum, bias and residual, is off by at most
        (C / 8 + 32) 2^-23 of the sum of magnitudes.  Activations stretch it by at most 1.13, and
        add, as evaluated, 2^-20 of their value (fp32 outputs: 64 2^-23; GELU: (x^2 + 14) 2^-23) or
        (bf16 outputs) 5e-7 and, of the value, 2e-3 for GELU where |GELU(x)| < |x| / 700, 6e-5 else,
        and (|x| + 8) 2^-23 for SiLU.  Then y is rounded to its type."""
        u = v @ self.w.T
        size = np.abs(v) @ np.abs(self.w).T
        if self.bias is not None:
            b = self.bias.double().cpu().numpy()
            u, size = u + b, size + np.abs(b)
        if res is not None:
            r = res.double().cpu().numpy()
            u, size = u + r, size + np.abs(r)
        tol = (self.C / 8 + 32) * 2.0 ** -23 * size
        y = R.act(u, self.act)
        if self.act == 3:
            tol = 1.13 * tol + (np.abs(y) * (u * u + 14) * 2.0 ** -23 if self.y == F32 else
                                5e-7 + np.abs(y) * np.where(u < -3, 2e-3, 6e-5))
        elif self.act == 4:
            tol = 1.13 * tol + np.abs(y) * ((np.abs(u) + 8) * 2.0 ** -23 if self.y == BF16 else
                                            2.0 ** -20)
        return y, tol + np.abs(y) * (2.0 ** -8 if self.y == BF16 else 2.0 ** -24) + 1e-38

    def check(self, M, **kw):
        x, v = self.input(M)
        res = self.res(M)
        out = self.layer(x, bias=self.bias, residual=res, **kw)
        _sync(self.torch, self.B)
        y, tol = self.expect(v, res)
        diff = np.abs(out.double().cpu().numpy() - y)
        assert (diff <= tol).all(), (diff / tol).max()
        return out


ROWS = [1, 2, 7, 8, 9, 16, 17, 31, 64, 65, 130, 300]


@pytest.mark.parametrize("C,K", [(1, 1), (32, 16), (127, 129), (128, 128), (130, 257), (1000, 333),
                                 (1456, 1111), (4096, 200)])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
def test_sizes(C, K, group):
    case = Case(C, K, group, zeros=group != 64, scale=F32 if group == 32 else BF16)
    for M in ROWS:
        case.check(M)


@pytest.mark.parametrize("x,x_group", [(BF16, 0), (F32, 0), (E4M3, 0), (E4M3, 128), (INT8, 0),
                                       (INT8, 128)])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("scale", [BF16, F32])
def test_types(x, x_group, group, scale):
    for C, K in ((300, 200), (1153, 515)):
        case = Case(C, K, group, x, F32, scale=scale, x_group=x_group, residual=True)
        for M in (1, 5, 16, 33, 100, 257):
            case.check(M)


@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("y", [BF16, F32])
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True),
                                           (True, True)])
def test_epilogues(act, y, bias, residual):
    case = Case(512, 272, 128, F32 if y == F32 else BF16, y, act=act, bias=bias, residual=residual)
    for M in (1, 12, 40, 256):
        case.check(M)


@pytest.mark.parametrize("M,C,K,x,group,x_group", [
    (1, 16384, 64, BF16, 128, 0), (8, 13000, 48, BF16, 32, 0), (8, 16384, 40, F32, 128, 0),
    (16, 8192, 130, E4M3, 64, 128), (16, 4096, 300, F32, 0, 0), (24, 16384, 33, BF16, 128, 0),
    (64, 8192, 1024, BF16, 64, 0), (128, 9000, 256, E4M3, 0, 128), (100, 16000, 130, INT8, 32, 0),
    (200, 4096, 128, F32, 32, 0), (256, 8192, 200, E4M3, 128, 128), (1, 2048, 9000, F32, 32, 0),
    (3, 100, 30000, BF16, 0, 0), (2, 700, 5000, INT8, 64, 128)])
def test_long_reductions_and_wide_layers(M, C, K, x, group, x_group):
    """Reductions split over warps, blocks and clusters; more outputs than fill the GPU once."""
    Case(C, K, group, x, F32, x_group=x_group, residual=True).check(M)


@pytest.mark.parametrize("M,C,K,x,group,x_group", [
    (3000, 256, 2500, BF16, 128, 0), (5000, 384, 640, E4M3, 64, 128), (2100, 320, 3000, F32, 32, 0),
    (9000, 130, 1000, INT8, 0, 128), (20000, 64, 300, BF16, 0, 0), (1100, 896, 2050, E4M3, 128, 0),
    (2049, 200, 2048, BF16, 32, 0), (700, 1024, 1100, INT8, 128, 128)])
def test_many_tiles(M, C, K, x, group, x_group):
    """More tiles than blocks: each of them takes several, its rings and accumulators go on."""
    Case(C, K, group, x, BF16, x_group=x_group, act=4).check(M)


# (rows, outputs): tiles of 64 rows; of 128, and of 128 in pairs of CTAs; of 160, and in pairs
WIDTHS = [(100, 600), (192, 4096), (500, 5000), (320, 4000), (639, 4790)]


@pytest.mark.parametrize("M,K", WIDTHS)
@pytest.mark.parametrize("group,x,x_group", [(0, BF16, 0), (128, BF16, 0), (64, BF16, 0),
                                             (32, F32, 0), (128, F32, 0), (0, INT8, 128),
                                             (64, INT8, 128), (32, E4M3, 128), (128, E4M3, 0)])
def test_every_tile_width(M, K, group, x, x_group):
    Case(1500, K, group, x, BF16, x_group=x_group, residual=True, act=1).check(M)


@pytest.mark.parametrize("M,x", [(1, BF16), (3, F32), (1, INT8)])
def test_rows_that_shared_memory_does_not_hold(M, x):
    Case(120001, 33, 128, x, F32, x_group=128 if x == INT8 else 0).check(M)


def test_more_rows_than_a_grid_has_blocks():
    """Of a layer so small that its rows would go to blocks 16 at a time."""
    Case(5, 7, 0, BF16, F32).check(16 * 65535 + 7)


@pytest.mark.parametrize("M", [1, 8, 16, 40])
@pytest.mark.parametrize("fmt", [E4M3, INT8])
def test_every_8_bit_code_times_every_weight(fmt, M):
    """A row holds one code, at a column of its own; the scales are 1, so y is exact."""
    torch, B, q8, W4Linear = _mods()
    C, K = 128, 256
    codes = torch.arange(K, dtype=torch.uint8) % 16  # of output k; its zero is k // 16
    layer = W4Linear(C, K, 128, x_dtype=None, x_q8=fmt, y_dtype=torch.float32,
                     scale_dtype=torch.float32)
    layer.load((codes * 17).reshape(K, 1).expand(K, C // 2).contiguous().cuda(),
               torch.ones(K, 1, device="cuda"),
               (torch.arange(K) // 16).to(torch.uint8).reshape(K, 1).cuda())
    weight = codes.double() - torch.arange(K).div(16, rounding_mode="floor").double()
    x = torch.arange(256, dtype=torch.uint8)
    value = x.view(torch.float8_e4m3fn if fmt == E4M3 else torch.int8).double()
    held = [i for i in range(256) if value[i] == value[i]]  # E4M3 has two NaNs
    while len(held) % M:
        held.append(held[-1])
    for start in range(0, len(held), M):
        rows = held[start:start + M]
        matrix = torch.zeros(M, C, dtype=torch.uint8)
        for m, i in enumerate(rows):
            matrix[m, (37 * i + i // 64) % C] = i
        t = q8.Q8Tensor(M, C, fmt, 0, matrix.cuda(), torch.ones(M, device="cuda"))
        y = layer(t)
        _sync(torch, B)
        assert torch.equal(y.double().cpu() + 0, torch.outer(value[rows], weight) + 0), start


def test_weights_past_32_bits():
    """More than 4 GB of packed weights: the first and the last outputs."""
    torch, B, q8, W4Linear = _mods()
    C, K, some = 16384, 540100, 100
    layer = W4Linear(C, K, 128, y_dtype=torch.float32)
    gen = torch.Generator(device="cuda").manual_seed(3)
    codes = torch.randint(0, 256, (K, C // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = (torch.rand(K, C // 128, generator=gen, device="cuda") / 128).bfloat16()
    zeros = torch.randint(0, 16, (K, C // 128), generator=gen, device="cuda", dtype=torch.uint8)
    layer.load(codes, scales, zeros)
    assert layer.w[0].numel() > 2 ** 32
    x = torch.randn(70, C, generator=gen, device="cuda").bfloat16()
    for M in (1, 70):
        y = layer(x[:M])
        _sync(torch, B)
        for at in (slice(0, some), slice(K - some, K)):
            q = torch.stack([codes[at] & 15, codes[at] >> 4], dim=2).reshape(some, C).double()
            w = (q - zeros[at].double().repeat_interleave(128, 1)) * \
                scales[at].double().repeat_interleave(128, 1)
            want, size = x[:M].double() @ w.t(), x[:M].double().abs() @ w.abs().t()
            # as Case.expect: sums, and y's rounding
            tol = (C / 8 + 32) * 2.0 ** -23 * size + want.abs() * 2.0 ** -24
            assert ((y[:, at].double() - want).abs() <= tol).all()


def test_tensors_of_a_load_on_another_stream_may_go():
    torch, B, q8, W4Linear = _mods()
    case = Case(2048, 512, 64)
    side = torch.cuda.Stream()
    x, _ = case.input(5)
    want = case.layer(x)
    layer = W4Linear(2048, 512, 64)
    side.wait_stream(torch.cuda.current_stream())
    codes, scales, zeros = (t.clone() for t in (case.codes, case.scales, case.zeros))
    side.wait_stream(torch.cuda.current_stream())
    layer.load(codes, scales, zeros, stream=side.cuda_stream)
    del codes, scales, zeros
    torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(layer(x), want)


def test_threads_share_a_layer():
    """Two threads, a stream each, calls of other sizes and strides."""
    import threading
    case = Case(700, 300, 64)
    torch = case.torch
    inputs = [torch.randn(M, 700 + pad, device="cuda").bfloat16()[:, :700]
              for M, pad in ((3, 0), (40, 4), (700, 0), (9, 100))]
    want = [case.layer(x) for x in inputs]
    torch.cuda.synchronize()
    wrong = []

    def work(order):
        stream = torch.cuda.Stream()
        for _ in range(20):
            for i in order:
                with torch.cuda.stream(stream):
                    y = case.layer(inputs[i])
                    if not torch.equal(y, want[i]):
                        wrong.append(i)

    threads = [threading.Thread(target=work, args=(o,)) for o in ((0, 1, 2, 3), (3, 2, 1, 0))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("M", [1, 11, 40, 150])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strided_rows_and_offsets(M, dtype):
    case = Case(200, 72, 64, dtype, dtype, residual=True)
    torch = case.torch
    x, v = case.input(M)
    res = case.res(M)
    y, tol = case.expect(v, res)
    for off, extra in ((0, 0), (1, 0), (0, 8), (3, 5), (8, 24)):
        def inside(rows, cols):
            flat = torch.full((off + rows * (cols + extra) + 7,), 55.0, dtype=case.y_dtype,
                              device="cuda")
            return flat, flat[off:off + rows * (cols + extra)].view(rows, cols + extra)[:, :cols]
        _, xs = inside(M, 200)
        _, rs = inside(M, 72)
        flat, ys = inside(M, 72)
        xs.copy_(x)
        rs.copy_(res)
        if M == 1:
            xs = xs.contiguous() if not off else xs
        out = case.layer(xs, bias=case.bias, residual=rs, out=ys)
        _sync(torch, case.B)
        assert out is ys
        assert (np.abs(out.double().cpu().numpy() - y) <= tol).all()
        kept = torch.ones_like(flat, dtype=torch.bool)
        kept[off:off + M * (72 + extra)].view(M, 72 + extra)[:, :72] = False
        assert (flat[kept] == 55).all()
        # into its residual
        again = case.layer(xs, bias=case.bias, residual=rs, out=rs)
        assert torch.equal(again, ys)


@pytest.mark.parametrize("M", [3, 13, 50, 200])
@pytest.mark.parametrize("x,x_group", [(BF16, 0), (F32, 0), (E4M3, 128), (INT8, 0)])
def test_bad_values_stay_in_their_rows(M, x, x_group):
    """Infinities and NaNs of x reach their own row's outputs and no others; rows do not depend
    on their neighbours."""
    case = Case(400, 150, 128, x, F32, x_group=x_group)
    torch = case.torch
    a = torch.randn(M, 400, device="cuda")
    if x == BF16:
        a = a.bfloat16()
    put = (lambda t: t) if x in (BF16, F32) else (lambda t: case.q8.quantize(t, x, x_group))
    good = case.layer(put(a))
    b = a.clone()
    b[1, 7], b[2, 399] = float("inf"), float("nan")
    bad = case.layer(put(b))
    _sync(torch, case.B)
    rest = [m for m in range(M) if m not in (1, 2)]
    assert torch.equal(good[rest], bad[rest])
    assert not torch.isfinite(bad[1]).any() and torch.isnan(bad[2]).all()
    if M > 16:  # one after the other: the same rows in another place
        turned = case.layer(put(a.flip(0).contiguous()))
        assert torch.equal(turned.flip(0), good)


def test_fp32_inputs_keep_24_bits():
    """Weights of one and a scale of one: the sum is x itself, in all of fp32's range."""
    torch, B, q8, W4Linear = _mods()
    for M in (1, 40):
        x = torch.zeros(M, 32, device="cuda")
        for m in range(M):
            x[m, m % 32] = 1 + 2.0 ** -23 * (2 * m + 1)
        x[0, 0] = 3.4028234e38
        layer = W4Linear(32, 16, 32, torch.float32, torch.float32, scale_dtype=torch.float32)
        layer.load(torch.full((16, 16), 0x99, dtype=torch.uint8, device="cuda"),
                   torch.ones(16, 1, device="cuda"))
        y = layer(x)
        assert torch.equal(y, x.sum(1, keepdim=True).expand(M, 16))


def test_all_codes_and_zeros():
    """Every code under every zero, one input at a time."""
    torch, B, q8, W4Linear = _mods()
    for group in (32, 64, 128, 0):
        C = 256
        groups = C // group if group else 1
        q = np.tile(np.arange(C) % 16, (16, 1))
        z = np.tile(np.arange(16)[:, None], (1, groups)).astype(np.uint8)
        layer = W4Linear(C, 16, group, y_dtype=torch.float32)
        layer.load(torch.from_numpy(R.pack_weights(q)).cuda(),
                   torch.full((16, groups), 0.5, dtype=torch.bfloat16, device="cuda"),
                   torch.from_numpy(z).cuda())
        x = torch.eye(C, device="cuda").bfloat16()
        want = torch.from_numpy(0.5 * (q - np.arange(16)[:, None])).float().t().cuda()
        assert torch.equal(layer(x), want)
        for m in range(0, C, 5):
            assert torch.equal(layer(x[m:m + 1]), want[m:m + 1])


def test_no_rows_leading_dimensions_streams_and_determinism():
    case = Case(384, 96, 64, act=3)
    torch = case.torch
    assert case.layer(torch.empty(0, 384, dtype=torch.bfloat16, device="cuda")).shape == (0, 96)
    x = torch.randn(2, 30, 384, device="cuda").bfloat16()
    y = case.layer(x, bias=case.bias)
    assert y.shape == (2, 30, 96)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = case.layer(x, bias=case.bias, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(y, z)
    for M in (1, 16, 60):
        rows = x.view(-1, 384)[:M]
        first = case.layer(rows, bias=case.bias)
        for _ in range(20):
            assert torch.equal(case.layer(rows, bias=case.bias), first)


def test_captured_and_replayed():
    """Two graphs of one layer, with workspaces of their own, replayed beside eager calls."""
    case = Case(1000, 200, 128, F32, F32)
    torch = case.torch
    xs = [torch.randn(M, 1000, device="cuda") for M in (40, 300, 1)]
    graphs, outs = [], []
    for x in xs:
        case.layer(x, bias=case.bias)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(case.layer(x, bias=case.bias))
        graphs.append(g)
    for seed in range(3):
        torch.manual_seed(seed)
        for x in xs:
            x.copy_(torch.randn_like(x))
        for g in graphs:
            g.replay()
        for x, out in zip(xs, outs):
            assert torch.equal(out, case.layer(x, bias=case.bias))
    _sync(torch, case.B)


def test_other_weights_and_refusals():
    case = Case(256, 64, 64)
    torch, q8 = case.torch, case.q8
    x, v = case.input(20)
    before = case.layer(x)
    case.layer.load(case.codes, case.scales * 2, case.zeros)
    assert torch.equal(case.layer(x), before * 2)
    for args in ((x.float(),), (x[:, :255],), (x, torch.zeros(63, device="cuda")),
                 (x, torch.zeros(64, device="cuda").bfloat16()), (x.cpu(),),
                 (x, None, None, torch.empty(19, 64, dtype=torch.bfloat16, device="cuda")),
                 (x, None, None, torch.empty(20, 64, device="cuda")),
                 (x, None, torch.empty(20, 64, device="cuda"))):
        with pytest.raises(ValueError):
            case.layer(*args)
    eight = Case(256, 64, 64, E4M3, x_group=128)
    for t in (q8.quantize(x, "int8", 128), q8.quantize(x, "e4m3", 0),
              q8.quantize(x[:, :128].contiguous(), "e4m3", 128), x):
        with pytest.raises(ValueError):
            eight.layer(t)
    with pytest.raises(case.B.GbconvError):
        case.layer(x, residual=torch.zeros(20, 64, dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("fmt,x_group", [("e4m3", 0), ("e4m3", 128), ("int8", 0), ("int8", 128)])
@pytest.mark.parametrize("rows", [1, 12, 200])
def test_norm_and_layers_together(fmt, x_group, rows):
    """x' = x + z; h = Q(norm(x')); t = silu(h W1^T + b1); y = x' + Q(t) W2^T + b2, captured as a
    user would run it, against 64 bits over the matrices that the calls hand on."""
    torch, B, q8, W4Linear = _mods()
    from cnn_convolution_gemm_gb300.norm import ResidualNorm
    C, hidden = 320, 768
    up = Case(C, hidden, 64, fmt, F32, act=4, x_group=x_group)
    down = Case(hidden, C, 128, fmt, BF16, residual=True, x_group=x_group, seed=1)
    norm = ResidualNorm(C, pre=B.CONV_NORM_RMS, h_q8=fmt, h_group=x_group)
    x, z = (torch.randn(rows, C, device="cuda").bfloat16() for _ in range(2))
    held = q8.empty(rows, hidden, fmt, "cuda", x_group)

    def run():
        x1, h = norm(x, z)
        t = up.layer(h, bias=up.bias)
        q8.quantize(t, fmt, x_group, out=held)
        return x1, h, t, down.layer(held, bias=down.bias, residual=x1)

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x1, h, t, y = run()
    graph.replay()
    _sync(torch, B)

    def val(m):
        return q8.dequantize(m, torch.float32).double().cpu().numpy()

    got = t.double().cpu().numpy()
    want, tol = up.expect(val(h), None)
    # (values read back in fp32 are off by 2^-24, within the bound's 32 steps)
    assert (np.abs(got - want) <= tol).all()
    want, tol = down.expect(val(held), x1)
    assert (np.abs(y.double().cpu().numpy() - want) <= tol).all()
    # the whole of it: within the two quantisations' steps
    d = (x.float() + z.float()).double().cpu().numpy()
    n = d / np.sqrt((d * d).mean(axis=1, keepdims=True) + 1e-6)
    u = n @ up.w.T + up.bias.double().cpu().numpy()
    ref = d + R.act(u, 4) @ down.w.T + down.bias.double().cpu().numpy()
    e = y.double().cpu().numpy() - ref
    assert np.sqrt((e * e).mean() / (ref * ref).mean()) < 2.0 ** -4
