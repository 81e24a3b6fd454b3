"""Refusals and sizes of the 4-bit and norm entry points (no GPU: everything here returns
before anything is launched), and the reference of their GPU tests against itself."""
import numpy as np
import pytest

from tests import fp4_ref as R


@pytest.fixture(scope="module")
def B():
    from cnn_convolution_gemm_gb300 import build
    build.build()
    from cnn_convolution_gemm_gb300 import binding
    binding.load_library()
    return binding


def refused(B, status, fn, *args, **kw):
    with pytest.raises(B.GbconvError) as e:
        fn(*args, **kw)
    assert e.value.status_name == status, (e.value.status_name, e.value.detail)
    assert e.value.detail


BAD, UNSUP, ALIGN, WS = ("CONV_ERR_BAD_PARAM", "CONV_ERR_UNSUPPORTED", "CONV_ERR_ALIGNMENT",
                         "CONV_ERR_WORKSPACE")
P = 0x10000  # a 16-byte aligned address that nothing dereferences


def test_sizes(B):
    assert B.conv_fp4_size(B.CONV_FP4_MX, 1, 1) == (16, 512)
    assert B.conv_fp4_size(B.CONV_FP4_MX, 129, 128) == (129 * 64, 2 * 512)
    assert B.conv_fp4_size(B.CONV_FP4_NV, 129, 129) == (129 * 80, 2 * 3 * 512)
    assert B.conv_fp4_size(B.CONV_FP4_NV, 0, 64) == (0, 0)
    # past 32 bits
    assert B.conv_fp4_size(B.CONV_FP4_MX, 1 << 20, 1 << 14) == (1 << 33, 1 << 29)
    refused(B, UNSUP, B.conv_fp4_size, B.CONV_FP4_MX, (1 << 30) + 1, 4)
    refused(B, UNSUP, B.conv_fp4_quantize, B.CONV_FP4_MX, B.CONV_BF16, 4, (1 << 30) + 1, P, 0, 1.0, P, P)
    refused(B, UNSUP, B.conv_fp4_create, B.CONV_FP4_MX, (1 << 30) + 1, 64)
    refused(B, BAD, B.conv_fp4_size, 2, 4, 4)
    refused(B, BAD, B.conv_fp4_size, B.CONV_FP4_MX, -1, 4)
    refused(B, BAD, B.conv_fp4_size, B.CONV_FP4_MX, 4, 0)


def test_quantize_refusals(B):
    q, dq = B.conv_fp4_quantize, B.conv_fp4_dequantize
    MX, NV, BF = B.CONV_FP4_MX, B.CONV_FP4_NV, B.CONV_BF16
    refused(B, BAD, q, 5, BF, 4, 64, P, 64, 1.0, P, P)
    refused(B, BAD, q, MX, B.CONV_INT8, 4, 64, P, 64, 1.0, P, P)
    refused(B, BAD, q, MX, BF, 4, 64, P, 63, 1.0, P, P)
    refused(B, BAD, q, MX, BF, -4, 64, P, 64, 1.0, P, P)
    refused(B, BAD, q, MX, BF, 4, 64, 0, 64, 1.0, P, P)
    refused(B, BAD, q, MX, BF, 4, 64, P, 64, 0.5, P, P)   # MX has no tensor scale
    for g in (0.0, -1.0, float("nan"), float("inf"), 1e-31, 1e31):
        refused(B, BAD, q, NV, BF, 4, 64, P, 64, g, P, P)
        refused(B, BAD, dq, NV, BF, 4, 64, P, P, g, P, 64)
    refused(B, ALIGN, q, MX, BF, 4, 64, P + 1, 64, 1.0, P, P)
    refused(B, ALIGN, q, MX, B.CONV_F32, 4, 64, P + 2, 64, 1.0, P, P)
    refused(B, ALIGN, q, MX, BF, 4, 64, P, 64, 1.0, P + 8, P)
    refused(B, ALIGN, dq, MX, BF, 4, 64, P, P + 8, 1.0, P, 64)
    refused(B, BAD, B.conv_fp4_pack_scales, MX, 4, 0, P, P)
    refused(B, BAD, B.conv_fp4_pack_scales, MX, 4, 64, 0, P)
    refused(B, ALIGN, B.conv_fp4_pack_scales, MX, 4, 64, P + 1, P + 1)
    # nothing to do: no tensor is looked at
    q(MX, BF, 0, 64, 0, 64, 1.0, 0, 0)
    dq(NV, BF, 0, 64, 0, 0, 0.5, 0, 64)
    B.conv_fp4_pack_scales(MX, 0, 64, 0, 0)


def test_product_refusals(B):
    MX, NV = B.CONV_FP4_MX, B.CONV_FP4_NV
    refused(B, BAD, B.conv_fp4_create, 7, 64, 64)
    refused(B, BAD, B.conv_fp4_create, MX, 0, 64)
    refused(B, BAD, B.conv_fp4_create, MX, 64, -1)
    refused(B, BAD, B.conv_fp4_create, MX, 64, 64, 3)
    d = B.conv_fp4_create(NV, 96, 48)
    refused(B, BAD, B.conv_fp4_set_epilogue, d, 5, False)
    refused(B, BAD, B.conv_fp4_set_tensor_scales, d, 0.0, 1.0, 1.0)
    refused(B, BAD, B.conv_fp4_set_tensor_scales, d, 1e30, 1e30, 1.0)
    refused(B, BAD, B.conv_fp4_set_strides, d, 95, 0, 0)
    refused(B, BAD, B.conv_fp4_set_strides, d, 0, 47, 0)
    refused(B, BAD, B.conv_fp4_set_strides, d, 0, 0, 47)
    refused(B, BAD, B.conv_fp4_workspace_size, d, -1)
    need = B.conv_fp4_workspace_size(d, 200)
    assert need >= sum(B.conv_fp4_size(NV, 200, 96))
    f = B.conv_fp4_fwd
    refused(B, BAD, f, d, -1, P, None, P, P, None, None, P, None, P, need)
    refused(B, UNSUP, f, d, (1 << 30) + 1, P, None, P, P, None, None, P, None, P, 1 << 60)
    refused(B, BAD, f, d, 200, None, None, P, P, None, None, P, None, P, need)
    refused(B, BAD, f, d, 200, P, P, P, P, None, None, P, None, P, need)      # scales of a float x
    refused(B, BAD, f, d, 200, P, None, P, P, None, None, P, P, P, need)      # scales of a float y
    refused(B, BAD, f, d, 200, P, None, P, P, None, P, P, None, P, need)      # residual not declared
    refused(B, WS, f, d, 200, P, None, P, P, None, None, P, None, None, 0)
    refused(B, WS, f, d, 200, P, None, P, P, None, None, P, None, P, need - 1)
    refused(B, ALIGN, f, d, 200, P + 1, None, P, P, None, None, P, None, P, need)
    refused(B, ALIGN, f, d, 200, P, None, P + 8, P, None, None, P, None, P, need)
    refused(B, ALIGN, f, d, 200, P, None, P, P, P + 2, None, P, None, P, need)
    refused(B, ALIGN, f, d, 200, P, None, P, P, None, None, P, None, P + 4, need)
    f(d, 0, None, None, None, None, None, None, None, None)  # no rows
    B.conv_fp4_destroy(d)
    c = B.conv_fp4_create(MX, 96, 48, B.CONV_FP4_IO_CODES, B.CONV_FP4_IO_CODES)
    refused(B, UNSUP, B.conv_fp4_set_epilogue, c, 0, True)
    refused(B, UNSUP, B.conv_fp4_set_strides, c, 100, 0, 0)
    refused(B, UNSUP, B.conv_fp4_set_strides, c, 0, 0, 100)
    refused(B, BAD, B.conv_fp4_set_tensor_scales, c, 2.0, 1.0, 1.0)
    refused(B, BAD, f, c, 8, P, None, P, P, None, None, P, P, P, 1 << 20)     # codes without scales
    refused(B, ALIGN, f, c, 8, P + 2, P, P, P, None, None, P, P, P, 1 << 20)
    B.conv_fp4_destroy(c)
    # the activations of the 4-bit product stay refused where convolutions do not have them
    conv = B.conv_desc_create(1, 8, 8, 8, 8, 3, 3, 1, 1)
    refused(B, BAD, B.conv_desc_set_epilogue, conv, B.CONV_ACT_GELU, False)
    B.conv_desc_destroy(conv)


def test_norm_refusals(B):
    refused(B, BAD, B.conv_norm_create, 0)
    refused(B, UNSUP, B.conv_norm_create, 32769)
    refused(B, BAD, B.conv_norm_create, 64, B.CONV_INT8)
    d = B.conv_norm_create(64)
    refused(B, BAD, B.conv_norm_set_post, d, 3)
    refused(B, BAD, B.conv_norm_set_post, d, B.CONV_NORM_RMS, -1.0)
    refused(B, BAD, B.conv_norm_set_pre, d, B.CONV_NORM_RMS, float("nan"))
    refused(B, BAD, B.conv_norm_set_pre, d, B.CONV_NORM_NONE, 0.0, P)
    refused(B, UNSUP, B.conv_norm_set_pre, d, B.CONV_NORM_RMS, 0.0, P, P)
    refused(B, ALIGN, B.conv_norm_set_pre, d, B.CONV_NORM_RMS, 0.0, P + 2)
    refused(B, BAD, B.conv_norm_set_gate, d, 3)
    refused(B, BAD, B.conv_norm_set_gate, d, 1, 0)
    refused(B, BAD, B.conv_norm_set_gate, d, 1, 1, float("inf"))
    refused(B, BAD, B.conv_norm_set_output, d, 3)
    refused(B, BAD, B.conv_norm_set_output, d, B.CONV_NORM_OUT_FP4_MX, 0.5)
    refused(B, BAD, B.conv_norm_set_output, d, B.CONV_NORM_OUT_FP4_NV, 0.0)
    refused(B, BAD, B.conv_norm_set_strides, d, 63)
    f = B.conv_norm_fwd
    refused(B, BAD, f, d, -1, P, P, None, P, None)
    refused(B, BAD, f, d, 4, None, P, None, P, None)
    refused(B, BAD, f, d, 4, P, P, None, None, None)      # nothing to write
    refused(B, BAD, f, d, 4, P, P, None, P, P)            # h without a norm before
    refused(B, BAD, f, d, 4, P, P, P, P, None)            # a gate that is not declared
    refused(B, ALIGN, f, d, 4, P + 1, P, None, P, None)
    B.conv_norm_set_pre(d, B.CONV_NORM_RMS)
    B.conv_norm_set_gate(d, B.CONV_GATE_SIGMOID)
    refused(B, BAD, f, d, 4, P, P, P, P, None)            # no h
    refused(B, BAD, f, d, 4, P, P, None, P, P)            # no gate
    refused(B, BAD, f, d, 4, P, P, P, P, P, P)            # scales of a float h
    B.conv_norm_set_output(d, B.CONV_NORM_OUT_FP4_MX)
    refused(B, BAD, f, d, 4, P, P, P, P, P)               # no scales of a 4-bit h
    refused(B, ALIGN, f, d, 4, P, P, P, P, P + 2, P)
    B.conv_norm_set_strides(d, 80, 0, 0, 72, 0)
    refused(B, BAD, f, d, 4, P, P, P, P, P, P)            # in place with another stride
    B.conv_norm_set_strides(d, 0, 0, 0, 0, 80)
    refused(B, UNSUP, f, d, 4, P, P, P, P, P, P)          # 4-bit rows are contiguous
    f(d, 0, None, None, None, None, None)
    B.conv_norm_destroy(d)


def test_block_refusals(B):
    MX, RMS, CODES = B.CONV_FP4_MX, B.CONV_NORM_RMS, B.CONV_FP4_IO_CODES

    def norm(C=64, out=B.CONV_NORM_OUT_FLOAT, **kw):
        d = B.conv_norm_create(C, **kw)
        B.conv_norm_set_pre(d, RMS)
        if out:
            B.conv_norm_set_output(d, out)
        return d
    n_in, n_out = norm(out=B.CONV_NORM_OUT_FP4_MX), norm()
    fc1, fc2 = B.conv_fp4_create(MX, 64, 96, CODES, CODES), B.conv_fp4_create(MX, 96, 64, CODES)
    make = B.conv_fp4_block_create
    refused(B, BAD, make, None, fc1, fc2, n_out)
    refused(B, BAD, make, n_in, fc2, fc1, n_out)                           # widths
    refused(B, BAD, make, norm(), fc1, fc2, n_out)                         # h not in 4 bits
    refused(B, BAD, make, norm(out=B.CONV_NORM_OUT_FP4_NV), fc1, fc2, n_out)
    refused(B, BAD, make, n_in, B.conv_fp4_create(MX, 64, 96, CODES), fc2, n_out)
    refused(B, BAD, make, n_in, fc1, B.conv_fp4_create(MX, 96, 64, CODES, B.CONV_FP4_IO_F32), n_out)
    refused(B, BAD, make, n_in, fc1, fc2, norm(x_dtype=B.CONV_F32))
    d = make(n_in, fc1, fc2, n_out)
    fwd, size = B.conv_fp4_block_fwd, B.conv_fp4_block_workspace_size
    # h 5 x 64 and t 5 x 96 (codes of 160 and 240 bytes, one row of scale tiles each), z: each
    # from a 256-byte boundary
    assert size(d, 5) == 256 + 512 + 256 + 512 + 768 and size(d, 0) == 0
    refused(B, BAD, size, d, -1)
    refused(B, UNSUP, size, d, (1 << 30) + 1)
    refused(B, BAD, fwd, d, 5, P, None, None, None, P, P, None, P, 1 << 20)      # no weights
    refused(B, BAD, B.conv_fp4_block_set_weights, d, P, None, None, P, P, None)
    refused(B, ALIGN, B.conv_fp4_block_set_weights, d, P, P + 8, None, P, P, None)
    refused(B, ALIGN, B.conv_fp4_block_set_weights, d, P, P, P + 2, P, P, None)
    B.conv_fp4_block_set_weights(d, P, P, None, P, P, None)
    fwd(d, 0, None, None, None, None, None, None, None, None, 0)
    refused(B, WS, fwd, d, 5, P, None, None, None, P, P, None, P, size(d, 5) - 1)
    refused(B, ALIGN, fwd, d, 5, P, None, None, None, P, P, None, P + 8, 1 << 20)
    refused(B, BAD, fwd, d, 5, P, P, None, None, P, P, None, P, 1 << 20)         # h without scales
    refused(B, BAD, fwd, d, 5, P, None, None, P, P, P, None, P, 1 << 20)         # a gate without need
    refused(B, BAD, fwd, d, 5, P, None, None, None, P, P, P, P, 1 << 20)         # scales of a float h
    refused(B, BAD, fwd, d, 5, None, None, None, None, P, P, None, P, 1 << 20)
    # a descriptor changed afterwards
    B.conv_fp4_set_epilogue(fc2, 0, 1)
    refused(B, BAD, fwd, d, 5, P, None, None, None, P, P, None, P, 1 << 20)
    B.conv_fp4_set_epilogue(fc2, 0, 0)
    B.conv_norm_set_strides(n_in, 70)
    refused(B, BAD, fwd, d, 5, P, None, None, None, P, P, None, P, 1 << 20)
    B.conv_fp4_block_destroy(d)


def test_reference_rounding():
    """The tests' own reference: levels, ties and saturation of E2M1 and E4M3."""
    v = np.array([0.25, 0.2501, 0.75, 0.7499, 1.25, 1.75, 2.5, 3.5, 5.0, 5.001, 7.0, -0.3, -9.0])
    want = [0, 0.5, 1, 0.5, 1, 2, 2, 4, 4, 6, 6, -0.5, -6]
    np.testing.assert_array_equal(R.e2m1_value(R.e2m1_code(v)), want)
    np.testing.assert_array_equal(R.e2m1_code(R.e2m1_value(np.arange(8, dtype=np.uint8))), np.arange(8))
    assert R.E4M3[-1] == 448 and R.E4M3[1] == 2.0 ** -9 and R.E4M3[8] == 2.0 ** -6
    np.testing.assert_array_equal(R.e4m3_byte(R.E4M3), np.arange(127))
    assert R.e4m3_value(R.e4m3_byte([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10])).tolist() == [16, 20, 0, 2.0 ** -8]
    # every MX block's largest element keeps 4 <= |x| / scale < 8
    x = np.abs(np.random.default_rng(0).standard_normal((50, 64))).astype(np.float32)
    code, byte = R.quantize(x, R.MX)
    s = R.scale_values(byte, R.MX)
    ratio = x.reshape(50, 2, 32).max(2) / s
    assert ((4 <= ratio) & (ratio < 8)).all()


def test_torch_layers_check_their_tensors(B):
    torch = pytest.importorskip("torch")
    from cnn_convolution_gemm_gb300 import fp4
    from cnn_convolution_gemm_gb300.norm import ResidualNorm
    with pytest.raises(ValueError):
        fp4.rows_of(torch.zeros(4, 6).t(), 4, "x")       # columns not contiguous
    with pytest.raises(ValueError):
        fp4.rows_of(torch.zeros(2, 3, 4)[:, :, :3], 3, "x")
    with pytest.raises(ValueError):
        fp4.rows_of(torch.zeros(1, 6).expand(4, 6), 6, "x")  # rows that overlap
    assert fp4.rows_of(torch.zeros(5, 9)[:, 2:8], 6, "x") == (5, 9)
    assert fp4.rows_of(torch.zeros(2, 3, 4), 4, "x") == (6, 4)
    layer = fp4.Fp4Linear(64, 32)
    with pytest.raises(RuntimeError):
        layer(torch.zeros(1, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        layer.load(torch.zeros(32, 33, dtype=torch.uint8), torch.zeros(32, 2, dtype=torch.uint8))
    with pytest.raises(ValueError):
        ResidualNorm(64, w_pre=torch.zeros(63), pre=B.CONV_NORM_RMS)
    with pytest.raises(ValueError):
        ResidualNorm(64, w_pre=torch.ones(64), pre=B.CONV_NORM_RMS)(
            torch.zeros(1, 64, dtype=torch.bfloat16))    # a tensor in host memory
    with pytest.raises(ValueError):
        fp4.quantize(torch.zeros(1, 64), B.CONV_FP4_MX)


# ---- the torch layers up to their launch, without a GPU -------------------------


@pytest.fixture
def host_layers(B, monkeypatch):
    """The torch layers over tensors in host memory that say they are on GPU 0, with launches
    that are only written down: (torch, fp4, up, calls, allocated).  Every buffer that the
    layers allocate is kept, so that addresses are not used twice."""
    torch = pytest.importorskip("torch")
    from cnn_convolution_gemm_gb300 import fp4

    class OnGpu(torch.Tensor):
        def get_device(self):
            return 0

    def up(t):
        return t.as_subclass(OnGpu)
    calls, allocated = [], []
    empty = torch.empty

    def kept_empty(*args, **kw):
        t = up(empty(*args, **kw))
        allocated.append(t)
        return t
    monkeypatch.setattr(torch, "empty", kept_empty)
    monkeypatch.setattr(fp4, "current_stream", lambda index: 7)
    monkeypatch.setattr(fp4, "current_device", lambda: 0, raising=False)
    for name in ("conv_fp4_fwd", "conv_fp4_block_fwd", "conv_norm_fwd", "conv_fp4_quantize",
                 "conv_fp4_dequantize", "conv_fp4_pack_scales"):
        monkeypatch.setattr(B, name, lambda *a, name=name: calls.append((name, a)))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return torch, fp4, up, calls, allocated


def _host_block(torch, up, **kw):
    from cnn_convolution_gemm_gb300.residual_block import Fp4ResidualBlock
    blk = Fp4ResidualBlock(64, 96, **kw)
    blk.prepack(up(torch.zeros(96, 64)), up(torch.zeros(64, 96)))
    return blk


@pytest.mark.parametrize("what", ["layer", "block"])
def test_captured_calls_have_workspaces_of_their_own(host_layers, monkeypatch, what):
    """A captured call's workspace is no other call's, before or after it; calls outside captures
    keep one, replaced by a larger one when it is too small."""
    torch, fp4, up, calls, allocated = host_layers
    if what == "layer":
        layer = fp4.Fp4Linear(64, 32)
        layer.prepack(up(torch.zeros(32, 64)))
    else:
        layer = _host_block(torch, up)

    def workspace(rows, capturing):
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
        layer(up(torch.zeros(rows, 64, dtype=torch.bfloat16)))
        name, args = calls[-1]
        at, size = (args[10], args[11]) if what == "layer" else (args[9], args[10])
        found = [t for t in allocated if t.data_ptr() <= at < t.data_ptr() + t.numel()]
        assert len(found) == 1 and at + size <= found[0].data_ptr() + found[0].numel()
        return id(found[0])
    small = workspace(20, False)
    captured = [workspace(20, True), workspace(20, True), workspace(300, True)]
    assert workspace(20, False) == small
    large = workspace(400, False)
    after = [workspace(20, True), workspace(400, False), workspace(300, False)]
    assert after[1] == after[2] == large != small
    captured.append(after[0])
    assert len({small, large, *captured}) == 6


def test_tensors_on_other_devices_are_refused(host_layers, monkeypatch):
    """Every tensor of a call in host memory, or on a GPU that the call does not run on, and every
    tensor that a layer keeps."""
    torch, fp4, up, calls, _ = host_layers
    from cnn_convolution_gemm_gb300 import binding as B
    from cnn_convolution_gemm_gb300.norm import ResidualNorm
    from cnn_convolution_gemm_gb300.residual_block import Fp4ResidualBlock
    RMS, LN, MX = B.CONV_NORM_RMS, B.CONV_NORM_LAYER, B.CONV_FP4_MX
    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8

    class OnOther(torch.Tensor):
        def get_device(self):
            return 1

    def here(*shape, dtype=bf):
        return up(torch.zeros(*shape, dtype=dtype))

    def elsewhere(t):
        host = torch.zeros(t.shape, dtype=t.dtype)
        return host, host.as_subclass(OnOther)

    def held(rows, cols, to=lambda t: t):
        cb, sb = B.conv_fp4_size(MX, rows, cols)
        return fp4.Fp4Tensor(rows, cols, MX, 1.0, to(here(cb, dtype=u8)), to(here(sb, dtype=u8)))

    def refused_elsewhere(call, **tensors):
        """call takes the tensors where they are, and none of them elsewhere."""
        call(**tensors)
        for name, t in tensors.items():
            for k in range(2):
                if isinstance(t, fp4.Fp4Tensor):
                    bad = held(t.rows, t.cols, lambda v, k=k: elsewhere(v)[k])
                else:
                    bad = elsewhere(t)[k]
                n = len(calls)
                with pytest.raises(ValueError):
                    call(**{**tensors, name: bad})
                assert len(calls) == n, name
    layer = fp4.Fp4Linear(64, 32, has_residual=True)
    layer.load(here(32, 32, dtype=u8), here(32, 2, dtype=u8))
    refused_elsewhere(layer, x=here(4, 64), bias=here(32, dtype=f32), residual=here(4, 32), out=here(4, 32))
    refused_elsewhere(layer.load, codes=here(32, 32, dtype=u8), scales=here(32, 2, dtype=u8))
    codes = fp4.Fp4Linear(64, 32, x_dtype=None, y_dtype=None)
    codes.load(here(32, 32, dtype=u8), here(32, 2, dtype=u8))
    refused_elsewhere(codes, x=held(4, 64), out=held(4, 32))
    refused_elsewhere(lambda x, out: fp4.quantize(x, MX, out=out), x=here(4, 64), out=held(4, 64))
    refused_elsewhere(lambda t, out: fp4.dequantize(t, out=out), t=held(4, 64), out=here(4, 64))
    with pytest.raises(ValueError):
        fp4.Fp4Tensor(4, 64, MX, 1.0, here(128, dtype=u8), torch.zeros(512, dtype=u8))
    with pytest.raises(ValueError):
        layer.load(*(here(32, n, dtype=u8).as_subclass(torch.Tensor) for n in (32, 2)))
    w = [here(64, dtype=f32) for _ in range(4)]
    for h_fmt in (None, MX):
        norm = ResidualNorm(64, post=LN, pre=LN, gate=B.CONV_GATE_LINEAR, h_fmt=h_fmt,
                            w_post=w[0], b_post=w[1], w_pre=w[2], b_pre=w[3])
        refused_elsewhere(norm, x=here(4, 64), z=here(4, 64), gate=here(4, 64), x_out=here(4, 64),
                          h_out=held(4, 64) if h_fmt is not None else here(4, 64))
    refused_elsewhere(ResidualNorm(64, pre=RMS), x=here(4, 64), h_out=here(4, 64))
    for t in elsewhere(w[0]):
        for i in range(4):
            with pytest.raises(ValueError):
                p = w[:i] + [t] + w[i + 1:]
                ResidualNorm(64, post=LN, pre=LN, w_post=p[0], b_post=p[1], w_pre=p[2], b_pre=p[3])
    for chain in (False, True):
        blk = _host_block(torch, up, gate=B.CONV_GATE_LINEAR, w_pre=w[0], w_post=w[1], w_next=w[2],
                          b1=here(96, dtype=f32), b2=here(64, dtype=f32), chain=chain)
        refused_elsewhere(blk, x=here(4, 64), gate=here(4, 64), h=held(4, 64), x_out=here(4, 64),
                          h_out=held(4, 64) if chain else here(4, 64))
    n = len(calls)
    for name, size in (("b1", 96), ("b2", 64), ("w_pre", 64), ("w_post", 64), ("w_next", 64)):
        for t in elsewhere(here(size, dtype=f32)):
            with pytest.raises(ValueError):
                _host_block(torch, up, **{name: t})(here(4, 64))
    assert not any(name == "conv_fp4_block_fwd" for name, _ in calls[n:])
    # all of it on a GPU that is not the current one
    monkeypatch.setattr(fp4, "current_device", lambda: 1)
    n = len(calls)
    for call in (lambda: layer(here(4, 64), residual=here(4, 32)), lambda: norm(here(4, 64)),
                 lambda: blk(here(4, 64), gate=here(4, 64)), lambda: fp4.quantize(here(4, 64), MX),
                 lambda: fp4.dequantize(held(4, 64)),
                 lambda: layer.load(here(32, 32, dtype=u8), here(32, 2, dtype=u8))):
        with pytest.raises(ValueError):
            call()
    assert len(calls) == n


@pytest.mark.parametrize("what", ["layer", "norm", "block", "part"])
def test_threads_share_a_layer(host_layers, monkeypatch, what):
    """Two threads whose tensors have other row strides: each launch finds its own.  A thread that
    has set its strides gives the other every chance to set others before it launches."""
    import threading
    torch, fp4, up, calls, _ = host_layers
    from cnn_convolution_gemm_gb300 import binding as B
    from cnn_convolution_gemm_gb300.norm import ResidualNorm
    if what == "layer":
        layer = fp4.Fp4Linear(64, 32)
        layer.load(up(torch.zeros(32, 32, dtype=torch.uint8)), up(torch.zeros(32, 2, dtype=torch.uint8)))
        run = [layer] * 2
    elif what == "norm":
        run = [ResidualNorm(64, pre=B.CONV_NORM_RMS)] * 2
    else:  # the block in both threads, or in one of them its norm behind
        blk = _host_block(torch, up)
        run = [blk, blk.norm_out if what == "part" else blk]
    now, seen = {}, {}
    meeting = threading.Barrier(2)

    def set_strides(desc, *strides):
        now[desc.value] = strides[0]
        try:
            meeting.wait(0.3)
        except threading.BrokenBarrierError:
            pass

    def launch(desc, *args):
        used = [blk.norm_in.desc, blk.norm_out.desc] if desc is getattr(run[0], "desc", None) and (
            what in ("block", "part")) else [desc]
        seen[threading.current_thread().name] = [now[d.value] for d in used]
    for name in ("conv_fp4_set_strides", "conv_norm_set_strides"):
        monkeypatch.setattr(B, name, set_strides)
    for name in ("conv_fp4_fwd", "conv_norm_fwd", "conv_fp4_block_fwd"):
        monkeypatch.setattr(B, name, launch)
    wide = [up(torch.zeros(4, ld, dtype=torch.bfloat16)) for ld in (72, 80)]
    threads = [threading.Thread(target=lambda i=i: run[i](wide[i][:, :64]), name=str(i)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert set(seen["0"]) == {72} and set(seen["1"]) == {80}, seen


def test_block_sets_the_strides_that_its_parts_leave(host_layers, monkeypatch):
    """What the descriptors of a block hold when it launches, after strided calls of each part."""
    torch, fp4, up, calls, _ = host_layers
    from cnn_convolution_gemm_gb300 import binding as B
    blk = _host_block(torch, up)
    now = {}
    for name in ("conv_fp4_set_strides", "conv_norm_set_strides"):
        monkeypatch.setattr(B, name, lambda desc, *strides: now.__setitem__(desc.value, strides))
    wide = lambda dtype=torch.bfloat16: up(torch.zeros(4, 80, dtype=dtype))[:, :64]  # noqa: E731
    h = blk.norm_in(wide(), x_out=wide())[1]
    z = blk.fc2(blk.fc1(h), out=wide(blk.fc2.y_dtype))
    blk.norm_out(wide(), z, x_out=wide(), h_out=wide())
    blk(up(torch.zeros(4, 64, dtype=torch.bfloat16)))
    assert now[blk.norm_in.desc.value] == (64,) * 5
    assert now[blk.fc2.desc.value] == (96, 64, 64)
    assert now[blk.norm_out.desc.value] == (64,) * 5


def test_type_of_z_alone(B):
    f = B.conv_norm_set_z_dtype
    d = B.conv_norm_create(64, B.CONV_BF16, B.CONV_BF16)
    f(d, B.CONV_F32)
    # z is aligned to its own element, gate and h to theirs
    B.conv_norm_set_gate(d, B.CONV_GATE_LINEAR)
    refused(B, ALIGN, B.conv_norm_fwd, d, 4, P, P + 2, P, P, None)
    refused(B, ALIGN, B.conv_norm_fwd, d, 4, P, P, P + 1, P, None)
    f(d, B.CONV_BF16)
    refused(B, BAD, f, d, B.CONV_INT8)
    refused(B, BAD, f, None, B.CONV_F32)
    B.conv_norm_destroy(d)
    for x, h, z in ((B.CONV_F32, B.CONV_BF16, B.CONV_F32), (B.CONV_F32, B.CONV_F32, B.CONV_BF16),
                    (B.CONV_BF16, B.CONV_F32, B.CONV_BF16)):
        d = B.conv_norm_create(64, x, h)
        refused(B, UNSUP, f, d, z)
        f(d, h)
        B.conv_norm_destroy(d)
    # a block's second layer gives what the norm behind takes
    CODES = B.CONV_FP4_IO_CODES
    n_in, n_out = B.conv_norm_create(64), B.conv_norm_create(64)
    B.conv_norm_set_pre(n_in, B.CONV_NORM_RMS)
    B.conv_norm_set_output(n_in, B.CONV_NORM_OUT_FP4_MX)
    fc1 = B.conv_fp4_create(B.CONV_FP4_MX, 64, 96, CODES, CODES)
    fc2 = B.conv_fp4_create(B.CONV_FP4_MX, 96, 64, CODES, B.CONV_FP4_IO_F32)
    refused(B, BAD, B.conv_fp4_block_create, n_in, fc1, fc2, n_out)
    f(n_out, B.CONV_F32)
    B.conv_fp4_block_destroy(B.conv_fp4_block_create(n_in, fc1, fc2, n_out))


@pytest.mark.parametrize("rows,cols", [(1, 1), (4, 64), (129, 65), (128, 4097), (0, 7)])
def test_fp4_tensors_have_their_bytes(B, rows, cols):
    torch = pytest.importorskip("torch")
    from cnn_convolution_gemm_gb300 import fp4
    for fmt in (B.CONV_FP4_MX, B.CONV_FP4_NV):
        cb, sb = B.conv_fp4_size(fmt, rows, cols)
        u8 = lambda n: torch.zeros(n, dtype=torch.uint8)  # noqa: E731
        t = fp4.Fp4Tensor(rows, cols, fmt, 1.0, u8(cb), u8(sb))
        assert t.shape == (rows, cols, fmt)
        fp4.Fp4Tensor(rows, cols, fmt, 1.0, u8(cb + 16), u8(sb + 16))
        bad = [(u8(2 * cb)[::2], u8(sb)), (u8(cb), u8(2 * sb)[::2]), (u8(cb).view(torch.int8), u8(sb)),
               (u8(cb - 1), u8(sb)), (u8(cb), u8(sb - 1))] if rows else []
        for codes, scales in bad:
            with pytest.raises(ValueError):
                fp4.Fp4Tensor(rows, cols, fmt, 1.0, codes, scales)


def test_other_types_are_refused(host_layers):
    torch, fp4, up, calls, _ = host_layers
    from cnn_convolution_gemm_gb300 import binding as B
    from cnn_convolution_gemm_gb300.norm import ResidualNorm
    half = torch.float16
    t = fp4.empty(4, 64, B.CONV_FP4_MX, "cpu")
    for call in (lambda: fp4.quantize(up(torch.zeros(4, 64, dtype=half)), B.CONV_FP4_MX),
                 lambda: fp4.dequantize(t, half), lambda: fp4.Fp4Linear(64, 32, x_dtype=half),
                 lambda: fp4.Fp4Linear(64, 32, y_dtype=half), lambda: ResidualNorm(64, half),
                 lambda: ResidualNorm(64, z_dtype=half), lambda: ResidualNorm(64, h_dtype=half)):
        with pytest.raises(ValueError):
            call()
    assert not calls
