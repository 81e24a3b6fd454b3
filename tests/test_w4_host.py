"""Refusals and sizes of the 8-bit matrices and of the layers with integer 4-bit weights (no
GPU: everything here returns before anything is launched), and the GPU tests' references
against themselves."""
import numpy as np
import pytest

from tests import w4_ref as R
from tests.test_fp4_host import ALIGN, BAD, UNSUP, WS, P, refused


@pytest.fixture(scope="module")
def B():
    from cnn_convolution_gemm_gb300 import build
    build.build()
    from cnn_convolution_gemm_gb300 import binding
    binding.load_library()
    return binding


def test_q8_sizes(B):
    E, I = B.CONV_Q8_E4M3, B.CONV_Q8_INT8
    assert B.conv_q8_size(E, 0, 1, 1) == (16, 4)
    assert B.conv_q8_size(I, 128, 5, 129) == (5 * 144, 5 * 2 * 4)
    assert B.conv_q8_size(E, 128, 0, 64) == (0, 0)
    assert B.conv_q8_size(E, 128, 1 << 20, 1 << 14) == (1 << 34, 1 << 29)  # past 32 bits
    refused(B, BAD, B.conv_q8_size, 2, 0, 4, 4)
    refused(B, BAD, B.conv_q8_size, E, 64, 4, 4)
    refused(B, BAD, B.conv_q8_size, E, 0, -1, 4)
    refused(B, BAD, B.conv_q8_size, E, 0, 4, 0)
    refused(B, UNSUP, B.conv_q8_size, E, 0, 4, (1 << 30) + 1)


@pytest.mark.parametrize("name", ["conv_q8_quantize", "conv_q8_dequantize"])
def test_q8_refusals(B, name):
    fn, dt = getattr(B, name), B.CONV_BF16

    def f(fmt, group, dtype, rows, cols, t, ld, codes, scales):
        if name == "conv_q8_quantize":
            fn(fmt, group, dtype, rows, cols, t, ld, codes, scales)
        else:
            fn(fmt, group, dtype, rows, cols, codes, scales, t, ld)
    refused(B, BAD, f, 2, 0, dt, 4, 4, P, 0, P, P)
    refused(B, BAD, f, 0, 32, dt, 4, 4, P, 0, P, P)
    refused(B, BAD, f, 0, 0, B.CONV_INT8, 4, 4, P, 0, P, P)
    refused(B, BAD, f, 0, 0, dt, -1, 4, P, 0, P, P)
    refused(B, BAD, f, 0, 0, dt, 4, 4, P, 3, P, P)
    refused(B, BAD, f, 0, 0, dt, 4, 4, None, 0, P, P)
    refused(B, BAD, f, 0, 0, dt, 4, 4, P, 0, None, P)
    refused(B, BAD, f, 0, 0, dt, 4, 4, P, 0, P, None)
    refused(B, UNSUP, f, 0, 0, dt, 4, (1 << 30) + 1, P, 0, P, P)
    refused(B, ALIGN, f, 0, 0, dt, 4, 4, P + 1, 0, P, P)
    refused(B, ALIGN, f, 0, 0, B.CONV_F32, 4, 4, P + 2, 0, P, P)
    refused(B, ALIGN, f, 0, 0, dt, 4, 4, P, 0, P + 8, P)
    refused(B, ALIGN, f, 0, 0, dt, 4, 4, P, 0, P, P + 4)
    f(0, 0, dt, 0, 4, None, 0, None, None)  # no rows


def test_w4_refusals(B):
    refused(B, BAD, B.conv_w4_create, 0, 64)
    refused(B, BAD, B.conv_w4_create, 64, -1)
    refused(B, UNSUP, B.conv_w4_create, (1 << 28) + 1, 64)
    refused(B, UNSUP, B.conv_w4_create, 64, 64, 16)
    refused(B, UNSUP, B.conv_w4_create, 64, 64, 256)
    refused(B, BAD, B.conv_w4_create, 64, 64, 128, B.CONV_INT8)
    refused(B, BAD, B.conv_w4_create, 64, 64, 128, B.CONV_BF16, 4)
    refused(B, BAD, B.conv_w4_create, 64, 64, 128, B.CONV_BF16, 0, B.CONV_INT8)
    d = B.conv_w4_create(2100, 48)
    refused(B, BAD, B.conv_w4_set_input_group, d, 64)
    refused(B, UNSUP, B.conv_w4_set_input_group, d, 128)  # bf16 x has no scales
    refused(B, BAD, B.conv_w4_set_epilogue, d, 5, False)
    refused(B, BAD, B.conv_w4_set_strides, d, 2099, 0, 0)
    refused(B, BAD, B.conv_w4_set_strides, d, 0, 47, 0)
    refused(B, BAD, B.conv_w4_set_strides, d, 0, 0, 47)
    refused(B, BAD, B.conv_w4_prepack, d, None, P, None, P)
    refused(B, BAD, B.conv_w4_prepack, d, P, None, None, P)
    refused(B, BAD, B.conv_w4_prepack, d, P, P, None, None)
    refused(B, ALIGN, B.conv_w4_prepack, d, P, P + 1, None, P)
    refused(B, ALIGN, B.conv_w4_prepack, d, P, P, None, P + 8)
    refused(B, BAD, B.conv_w4_workspace_size, d, -1)
    f, need = B.conv_w4_fwd, B.conv_w4_workspace_size(d, 200)
    assert need == 200 * 2104 * 2 and B.conv_w4_workspace_size(d, 1) == 0
    refused(B, BAD, f, d, -1, P, None, P, None, None, P)
    refused(B, UNSUP, f, d, (1 << 30) + 1, P, None, P, None, None, P)
    refused(B, BAD, f, d, 4, None, None, P, None, None, P)
    refused(B, BAD, f, d, 4, P, None, None, None, None, P)
    refused(B, BAD, f, d, 4, P, None, P, None, None, None)
    refused(B, BAD, f, d, 4, P, P, P, None, None, P)       # scales of a bf16 x
    refused(B, BAD, f, d, 4, P, None, P, None, P, P)       # a residual that is not declared
    refused(B, WS, f, d, 200, P, None, P, None, None, P, P, need - 1)
    refused(B, WS, f, d, 200, P, None, P, None, None, P, None, need)
    refused(B, ALIGN, f, d, 200, P, None, P, None, None, P, P + 4, need)
    refused(B, ALIGN, f, d, 4, P + 1, None, P, None, None, P)
    refused(B, ALIGN, f, d, 4, P, None, P + 8, None, None, P)
    refused(B, ALIGN, f, d, 4, P, None, P, P + 2, None, P)
    refused(B, ALIGN, f, d, 4, P, None, P, None, None, P + 1)
    B.conv_w4_set_epilogue(d, 0, True)
    refused(B, BAD, f, d, 4, P, None, P, None, None, P)    # no residual
    B.conv_w4_set_strides(d, 0, 64, 80)
    refused(B, BAD, f, d, 4, P, None, P, None, P, P)       # into it with another stride
    f(d, 0, None, None, None, None, None, None)            # no rows
    B.conv_w4_destroy(d)
    q = B.conv_w4_create(96, 48, 0, B.CONV_F32, B.CONV_W4_IO_INT8, B.CONV_F32)
    B.conv_w4_set_input_group(q, 128)
    refused(B, UNSUP, B.conv_w4_set_strides, q, 100, 0, 0)
    refused(B, BAD, f, q, 4, P, None, P, None, None, P)    # no scales
    refused(B, ALIGN, f, q, 4, P + 8, P, P, None, None, P)
    refused(B, ALIGN, B.conv_w4_prepack, q, P, P + 2, None, P)
    B.conv_w4_destroy(q)


def test_packed_sizes(B):
    def size(C, K, group, dtype):
        d = B.conv_w4_create(C, K, group, dtype)
        n = B.conv_w4_packed_size(d)
        B.conv_w4_destroy(d)
        return n
    # tiles of 128 x 128: codes, then zeros (a byte) and scales of each group
    assert size(128, 128, 128, B.CONV_BF16) == 8192 + 128 * 3
    assert size(129, 1, 32, B.CONV_F32) == 2 * (8192 + 128 * 4 * 5)
    assert size(4096, 4096, 0, B.CONV_BF16) == 32 * 32 * 8192 + 4096 * 3
    assert size(1 << 17, 1 << 17, 0, B.CONV_BF16) == (1 << 33) + (1 << 17) * 3  # past 32 bits


def test_norm_q8_refusals(B):
    d = B.conv_norm_create(64)
    refused(B, BAD, B.conv_norm_set_output_q8, d, 2)
    refused(B, BAD, B.conv_norm_set_output_q8, d, 0, 64)
    B.conv_norm_set_pre(d, B.CONV_NORM_RMS)
    B.conv_norm_set_output_q8(d, B.CONV_Q8_E4M3, 128)
    f = B.conv_norm_fwd
    refused(B, BAD, f, d, 4, P, P, None, P, P)             # no scales of an 8-bit h
    refused(B, ALIGN, f, d, 4, P, P, None, P, P + 2, P)
    refused(B, ALIGN, f, d, 4, P, P, None, P, P, P + 4)
    B.conv_norm_set_strides(d, 0, 0, 0, 0, 80)
    refused(B, UNSUP, f, d, 4, P, P, None, P, P, P)        # its rows are contiguous
    B.conv_norm_set_strides(d)
    B.conv_norm_set_output(d, B.CONV_NORM_OUT_FLOAT)       # and back
    refused(B, BAD, f, d, 4, P, P, None, P, P, P)
    B.conv_norm_destroy(d)


def test_a_4_bit_block_refuses_an_8_bit_norm(B):
    MX, CODES = B.CONV_FP4_MX, B.CONV_FP4_IO_CODES
    n_in, n_out = B.conv_norm_create(64), B.conv_norm_create(64)
    B.conv_norm_set_pre(n_in, B.CONV_NORM_RMS)
    B.conv_norm_set_output_q8(n_in, B.CONV_Q8_E4M3)
    f1 = B.conv_fp4_create(MX, 64, 128, CODES, CODES)
    f2 = B.conv_fp4_create(MX, 128, 64, CODES, B.CONV_FP4_IO_BF16)
    refused(B, BAD, B.conv_fp4_block_create, n_in, f1, f2, n_out)
    for d in (f1, f2):
        B.conv_fp4_destroy(d)
    for d in (n_in, n_out):
        B.conv_norm_destroy(d)


def test_torch_layers_check_their_tensors(B):
    import torch
    from cnn_convolution_gemm_gb300 import q8
    from cnn_convolution_gemm_gb300.norm import ResidualNorm
    from cnn_convolution_gemm_gb300.w4 import W4Linear
    u8, f32 = torch.uint8, torch.float32
    for make in (lambda: q8.empty(4, 64, "fp8", "cpu"), lambda: q8.empty(4, 64, "int8", "cpu", 64),
                 lambda: q8.Q8Tensor(4, 64, "int8", 0, torch.empty(255, dtype=u8), torch.empty(4)),
                 lambda: q8.Q8Tensor(4, 64, "int8", 0, torch.empty(256, dtype=u8), torch.empty(3)),
                 lambda: q8.Q8Tensor(4, 130, "int8", 128, torch.empty(4 * 144, dtype=u8),
                                     torch.empty(7)),
                 lambda: q8.Q8Tensor(4, 64, "int8", 0, torch.empty(256, dtype=f32), torch.empty(4)),
                 lambda: q8.Q8Tensor(4, 64, "int8", 0, torch.empty(512, dtype=u8)[::2],
                                     torch.empty(4)),
                 lambda: q8.Q8Tensor(4, 64, "int8", 0, torch.empty(272, dtype=u8)[8:],
                                     torch.empty(4)),
                 lambda: q8.quantize(torch.zeros(4, 64, dtype=torch.float16), "int8"),
                 lambda: q8.quantize(torch.zeros(4, 64), "int8"),               # not on a GPU
                 lambda: q8.quantize(torch.zeros(4, 64), "int8", out=q8.empty(4, 64, "e4m3", "cpu")),
                 lambda: q8.quantize(torch.zeros(1, 64).expand(4, 64), "int8"),
                 lambda: q8.dequantize(q8.empty(4, 64, "int8", "cpu"), out=torch.empty(3, 64)),
                 lambda: W4Linear(64, 64, x_dtype=None), lambda: W4Linear(64, 64, x_q8="int8"),
                 lambda: W4Linear(64, 64, x_dtype=torch.float16),
                 lambda: W4Linear(64, 64, x_dtype=None, x_q8="int4"),
                 lambda: ResidualNorm(64, h_q8="int4"), lambda: ResidualNorm(64, h_q8=0, h_group=1),
                 lambda: ResidualNorm(64, h_q8=0, h_fmt=B.CONV_FP4_MX)):
        with pytest.raises(ValueError):
            make()
    layer = W4Linear(65, 48, 32, scale_dtype=f32)
    codes, scales = torch.zeros(48, 33, dtype=u8), torch.zeros(48, 3)
    for args in ((codes[:, :32], scales), (codes.int(), scales), (codes, scales[:, :2]),
                 (codes, scales.bfloat16()), (codes, scales, torch.zeros(48, 2, dtype=u8)),
                 (codes, scales, torch.zeros(48, 3)), (codes, scales)):
        with pytest.raises(ValueError):
            layer.load(*args)
    with pytest.raises(RuntimeError):
        layer(torch.zeros(2, 65, dtype=torch.bfloat16))


def test_references():
    assert R.e4m3_values()[126] == 448 and R.e4m3_values()[1] == 2.0 ** -9
    x = np.array([[448.0, 17.0, 19.0, -18.0, 0.0, 2.0 ** -10, 3 * 2.0 ** -10]], np.float32)
    code, s = R.quantize(x, R.E4M3, 0)
    assert s[0, 0] == 1 and code.tolist() == [[448, 16, 20, -18, 0, 0, 2.0 ** -8]]
    # half the largest is next to 63.5, on either side of it as its scale was rounded
    for top in (1.0, 3.0, 100.0, 1.1):
        x = np.array([[top, top / 2]], np.float32)
        code, s = R.quantize(x, R.INT8, 0)
        exact = 254 * int(x[0, 1] * 2.0 ** 60)  # |x| <> 63.5 s in whole numbers
        assert code[0, 1] == (64 if exact >= int(127 * 127 * (float(s[0, 0]) * 2.0 ** 60)) else 63)
    q = np.arange(10)[None] % 16
    assert R.pack_weights(q).tolist() == [[0x10, 0x32, 0x54, 0x76, 0x98]]
    assert R.weights(q, np.full((1, 1), 0.5), None, 0)[0, 9] == 0.5
