"""What the 8-bit entry points refuse, without a GPU: the documented status before any CUDA call, and the
binding's own checks. Addresses are fake and never dereferenced."""
import ctypes

import pytest
import torch

import cnn_convolution_nhwc_b200 as cb

V = ctypes.c_void_p
X, R, W, H, Q, S = (V(i << 24) for i in range(1, 7))
Y, B, WS = V(7 << 24), V(8 << 24), V(9 << 24)
INV, UNS, MIS = cb.CONV_ERR_INVALID_ARG, cb.CONV_ERR_UNSUPPORTED, cb.CONV_ERR_MISALIGNED
BF16, F32 = cb.CONV_BF16, cb.CONV_F32


def off(p, n):
    return V(p.value + n)


def test_row_pitch():
    assert [cb.lib.conv_i8_row_pitch(c) for c in (1, 15, 16, 17, 33, 4096, 4097)] == [32, 32, 32, 32, 64, 4096, 4128]
    assert cb.lib.conv_i8_row_pitch(0) == 0 and cb.lib.conv_i8_row_pitch(-3) == 0
    assert cb.lib.conv_i8_row_pitch(2 ** 31 - 32) == 2 ** 31 - 32 and cb.lib.conv_i8_row_pitch(2 ** 31 - 1) == 0


@pytest.mark.parametrize("args,code", [
    # x, residual, weight, h, q, scale, M, C, ldq, eps, dtype
    ((None, R, W, H, Q, S, 2, 20, 32, 1e-6, BF16), INV),
    ((X, R, None, H, Q, S, 2, 20, 32, 1e-6, BF16), INV),
    ((X, R, W, None, Q, S, 2, 20, 32, 1e-6, BF16), INV),       # a residual without h
    ((X, None, W, H, Q, S, 2, 20, 32, 1e-6, BF16), INV),       # h without a residual
    ((X, R, W, H, None, S, 2, 20, 32, 1e-6, BF16), INV),
    ((X, R, W, H, Q, None, 2, 20, 32, 1e-6, BF16), INV),
    ((X, R, W, H, Q, S, 0, 20, 32, 1e-6, BF16), INV),
    ((X, R, W, H, Q, S, 2, 0, 32, 1e-6, BF16), INV),
    ((X, R, W, H, Q, S, 2, 20, 16, 1e-6, BF16), INV),          # rows overlap
    ((X, R, W, H, Q, S, 2, 20, 24, 1e-6, BF16), MIS),          # pitch off 16 bytes
    ((X, R, W, H, off(Q, 8), S, 2, 20, 32, 1e-6, BF16), MIS),
    ((X, R, W, H, Q, S, 2, 20, 32, 0.0, BF16), INV),
    ((X, R, W, H, Q, S, 2, 20, 32, float("nan"), BF16), INV),
    ((X, R, W, H, Q, S, 2, 20, 32, float("inf"), BF16), INV),
    ((X, R, W, H, Q, S, 2, 20, 32, 1e-6, 2), INV),
    ((off(X, 1), R, W, H, Q, S, 2, 20, 32, 1e-6, BF16), MIS),
    ((off(X, 2), R, W, H, Q, S, 2, 20, 32, 1e-6, F32), MIS),
    ((X, R, off(W, 2), H, Q, S, 2, 20, 32, 1e-6, BF16), MIS),
    ((X, R, W, off(X, 2), Q, S, 2, 20, 32, 1e-6, BF16), INV),  # h over x, not on it
    ((X, R, W, off(R, 40), Q, S, 2, 20, 32, 1e-6, BF16), INV),
    ((X, R, W, H, X, S, 2, 20, 32, 1e-6, BF16), INV),          # q on x
    ((X, R, W, H, H, S, 2, 20, 32, 1e-6, BF16), INV),          # q on h
    ((X, R, W, H, Q, off(Q, 48), 2, 20, 32, 1e-6, BF16), INV), # scale inside q
    ((X, R, W, H, Q, W, 2, 20, 32, 1e-6, BF16), INV),
])
def test_rmsnorm_rejects(args, code):
    assert cb.lib.rmsnorm_i8_fwd(*args, None) == code


@pytest.mark.parametrize("args,code", [
    # x, q, scale, M, C, ldq, glu, dtype
    ((None, Q, S, 2, 20, 32, 0, BF16), INV),
    ((X, Q, S, -1, 20, 32, 0, BF16), INV),
    ((X, Q, S, 2, 20, 32, 2, BF16), INV),
    ((X, Q, S, 2, 20, 32, 0, -1), INV),
    ((X, Q, S, 2, 20, 40, 0, BF16), MIS),
    ((X, off(X, 96), S, 2, 20, 32, 1, BF16), INV),   # inside the second half of the gated rows
    ((X, Q, off(X, 152), 2, 20, 32, 1, BF16), INV),
    ((X, Q, off(S, 2), 2, 20, 32, 0, BF16), MIS),
    ((X, Q, S, 1, 2 ** 27 + 1, 2 ** 27 + 16, 0, BF16), UNS),
])
def test_quant_rows_rejects(args, code):
    assert cb.lib.quant_rows_i8_fwd(*args, None) == code


@pytest.mark.parametrize("args,code", [
    # F, Wq, scale, Cin, Cout, ldw, dtype
    ((None, Q, S, 20, 8, 32, BF16), INV),
    ((X, Q, S, 0, 8, 32, BF16), INV),
    ((X, Q, S, 20, 8, 16, BF16), INV),
    ((X, Q, S, 20, 8, 33, BF16), MIS),
    ((X, Q, S, 131072, 8, 131072, BF16), UNS),
    ((X, X, S, 20, 8, 32, BF16), INV),
    ((X, Q, S, 20, 8, 32, 7), INV),
    ((off(X, 2), Q, S, 20, 8, 32, F32), MIS),
])
def test_quant_filter_rejects(args, code):
    assert cb.lib.quant_filter_i8_fwd(*args, None) == code


@pytest.mark.parametrize("args,code", [
    # q, scale, y, M, C, ldq, dtype
    ((None, S, Y, 2, 20, 32, BF16), INV),
    ((Q, S, Y, 2, 20, 20, BF16), MIS),
    ((Q, S, Q, 2, 20, 32, BF16), INV),
    ((Q, S, Y, 0, 20, 32, BF16), INV),
    ((Q, S, off(Y, 1), 2, 20, 32, BF16), MIS),
    ((Q, S, Y, 1, 2 ** 27 + 1, 2 ** 27 + 16, BF16), UNS),
])
def test_dequant_rejects(args, code):
    assert cb.lib.dequant_rows_i8_fwd(*args, None) == code


@pytest.mark.parametrize("args,code", [
    # q, q_scale, Wq, w_scale, bias, Y, M, Cin, Cout, ldq, ldw, dtype
    ((None, S, W, R, B, Y, 2, 20, 8, 32, 32, BF16), INV),
    ((Q, None, W, R, B, Y, 2, 20, 8, 32, 32, BF16), INV),
    ((Q, S, None, R, B, Y, 2, 20, 8, 32, 32, BF16), INV),
    ((Q, S, W, None, B, Y, 2, 20, 8, 32, 32, BF16), INV),
    ((Q, S, W, R, B, None, 2, 20, 8, 32, 32, BF16), INV),
    ((Q, S, W, R, B, Y, 0, 20, 8, 32, 32, BF16), INV),
    ((Q, S, W, R, B, Y, 2, 20, 0, 32, 32, BF16), INV),
    ((Q, S, W, R, B, Y, 2, 20, 8, 16, 32, BF16), INV),
    ((Q, S, W, R, B, Y, 2, 20, 8, 32, 40, BF16), MIS),
    ((off(Q, 4), S, W, R, B, Y, 2, 20, 8, 32, 32, BF16), MIS),
    ((Q, S, W, R, off(B, 1), Y, 2, 20, 8, 32, 32, BF16), MIS),
    ((Q, S, W, R, B, off(Y, 2), 2, 20, 8, 32, 32, F32), MIS),
    ((Q, S, W, R, B, Y, 2, 131072, 8, 131072, 131072, BF16), UNS),
    ((Q, S, W, R, B, Y, 2 ** 31 - 512, 20, 8, 32, 32, BF16), UNS),
    ((Q, S, W, R, B, Y, 2, 20, 2 ** 31 - 512, 32, 32, BF16), UNS),
    ((Q, S, W, R, B, Q, 2, 20, 8, 32, 32, BF16), INV),
    ((Q, S, W, R, Y, Y, 2, 20, 8, 32, 32, BF16), INV),
    ((Q, S, W, R, B, Y, 2, 20, 8, 32, 32, 5), INV),
])
def test_pointwise_rejects(args, code):
    assert cb.lib.pointwise_i8_fwd(*args, None) == code


@pytest.mark.parametrize("args,code", [
    # X, norm, eps, Wq, w_scale, bias, Y, workspace, bytes, N, H, W, Cin, Cout, ldw
    ((None, None, 0.0, W, R, B, Y, WS, 1 << 20, 1, 2, 3, 20, 8, 32), INV),
    ((X, None, 0.0, W, R, B, Y, None, 1 << 20, 1, 2, 3, 20, 8, 32), INV),
    ((X, None, 0.0, W, R, B, Y, WS, 6 * 36 - 1, 1, 2, 3, 20, 8, 32), INV),   # workspace too small
    ((X, H, 0.0, W, R, B, Y, WS, 1 << 20, 1, 2, 3, 20, 8, 32), INV),         # a norm needs eps
    ((X, None, 0.0, W, R, B, Y, off(WS, 4), 1 << 20, 1, 2, 3, 20, 8, 32), MIS),
    ((X, None, 0.0, W, R, B, Y, X, 1 << 20, 1, 2, 3, 20, 8, 32), INV),       # workspace on X
    ((X, None, 0.0, W, R, B, Y, W, 1 << 20, 1, 2, 3, 20, 8, 32), INV),       # ... on the filter
    ((X, None, 0.0, W, R, B, WS, WS, 1 << 20, 1, 2, 3, 20, 8, 32), INV),     # ... on Y
    ((X, None, 0.0, W, R, B, X, WS, 1 << 20, 1, 2, 3, 20, 8, 32), INV),
    ((X, None, 0.0, W, R, B, Y, WS, 1 << 20, 1, 0, 3, 20, 8, 32), INV),
    ((X, None, 0.0, W, R, B, Y, WS, 1 << 20, 1, 2, 3, 20, 8, 24), MIS),
    ((X, None, 0.0, W, R, B, Y, WS, 1 << 60, 4096, 4096, 4096, 20, 8, 32), UNS),
    ((X, None, 0.0, W, R, B, Y, WS, 1 << 60, 1, 2, 3, 131072, 8, 131072), UNS),
])
def test_layer_rejects(args, code):
    assert cb.lib.conv2d_nhwc_fwd_i8(*args, None) == code


def test_layer_workspace():
    assert cb.lib.conv2d_nhwc_i8_workspace(2, 3, 5, 20) == 30 * (32 + 4)
    assert cb.lib.conv2d_nhwc_i8_workspace(1, 1, 1, 16) == 36
    assert cb.lib.conv2d_nhwc_i8_workspace(0, 3, 5, 20) == 0
    assert cb.lib.conv2d_nhwc_i8_workspace(1, 1, 1, 131072) == 0
    assert cb.lib.conv2d_nhwc_i8_workspace(65536, 65536, 65536, 16) == 0


def test_binding_checks():
    x = torch.zeros(2, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        cb.quant_rows_i8_fwd(x)
    with pytest.raises(TypeError, match="bfloat16 or torch.float32"):
        cb.quant_rows_i8_fwd(x.half())
    with pytest.raises(TypeError, match="Tensor"):
        cb.rmsnorm_i8_fwd([1.0], torch.ones(1))
    with pytest.raises(ValueError, match="1 x 1"):
        cb.quant_filter_i8_fwd(torch.zeros(3, 3, 8, 8))
    with pytest.raises(TypeError, match="int8"):
        cb.dequant_rows_i8_fwd(x, torch.ones(2))
    with pytest.raises(ValueError, match="positive"):
        cb.empty_rows_i8(0, 8, device="cpu")
    e = cb.empty_rows_i8(3, 20, device="cpu")
    assert e.shape == (3, 20) and e.stride() == (32, 1)


def test_sizes_past_int_are_not_cut():
    with pytest.raises(ValueError, match="larger than 2"):
        cb.empty_rows_i8(2 ** 32 + 4, 8, device="meta")
    with pytest.raises(ValueError, match="larger than 2"):
        cb.empty_rows_i8(1, 2 ** 32 + 8, device="meta")
