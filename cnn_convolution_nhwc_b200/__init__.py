"""Forward 2-D convolution on B200 (sm_100a): thin Python binding of the C ABI.

The functions here only marshal arguments -- shape and dtype checks, output allocation
through PyTorch, the current CUDA stream -- and call the C entry points of
libconv_b200.so with the same names (declared in include/conv_b200.h). Every step of the
computation runs in the library's CUDA kernels; there is no CPU or PyTorch fallback, and
importing this package fails if the library cannot be loaded.

    conv2d_nhwc_fwd(X, F)        dense NHWC conv, bf16 [N,H,W,Cin] x [K,K,Cin,Cout] -> bf16
    conv2d_nhwc_fwd_f32(X, F)    the same with float32 tensors
    conv2d_nhwc_fwd_ex(X, F, b)  bf16 with stride, zero padding, dilation and a float32 bias
    depthwise_fwd(x, w, bias)    depthwise conv, float32 NCHW, exact or fast mode

In 8-bit integers (signed bytes with a float32 scale per row), the K = 1 convolution and what
feeds it:

    conv2d_nhwc_fwd_i8(X, Wq, w_scale, bias, norm)   dense 1 x 1 conv of bf16 X, quantised per pixel
    rmsnorm_i8_fwd(x, weight, residual)              norm (and residual addition) -> 8-bit rows
    quant_rows_i8_fwd(x, glu)                        rows, or silu(gate) * up, -> 8-bit rows
    quant_filter_i8_fwd(F)                           filter [Cin,Cout] -> 8-bit rows [Cout,Cin]
    pointwise_i8_fwd(q, q_scale, Wq, w_scale, bias)  their product
    dequant_rows_i8_fwd(q, scale)                    8-bit rows back to bf16 or float32
"""
from __future__ import annotations

import ctypes
import os

from . import build as _build

CONV_OK = 0
CONV_ERR_INVALID_ARG = -1
CONV_ERR_UNSUPPORTED = -2
CONV_ERR_MISALIGNED = -3
CONV_ERR_CUDA = -4
CONV_ERR_DEVICE_TIMEOUT = -5
CONV_ERR_DEVICE_BOUNDS = -6
DW_EXACT = 0
DW_FAST = 1
CONV_BF16 = 0
CONV_F32 = 1

# CONV_B200_DEBUG_BOUNDS=1 at import loads the bounds-checked build of the same library (every
# computed global access checked; a failure sets CONV_ERR_DEVICE_BOUNDS and skips the access)
DEBUG_BOUNDS = os.environ.get("CONV_B200_DEBUG_BOUNDS", "0") == "1"
LIB_PATH = _build.build(debug_bounds=DEBUG_BOUNDS)
lib = ctypes.CDLL(LIB_PATH)

_P = ctypes.c_void_p
_I = ctypes.c_int
lib.conv2d_nhwc_fwd.argtypes = [_P, _P, _P] + [_I] * 6 + [_P]
lib.conv2d_nhwc_fwd.restype = _I
lib.conv2d_nhwc_fwd_f32.argtypes = [_P, _P, _P] + [_I] * 6 + [_P]
lib.conv2d_nhwc_fwd_f32.restype = _I
lib.conv2d_nhwc_fwd_ex.argtypes = [_P, _P, _P, _P] + [_I] * 9 + [_P]
lib.conv2d_nhwc_fwd_ex.restype = _I
lib.conv2d_nhwc_fwd_grouped.argtypes = [_P, _P, _P, _P] + [_I] * 14 + [_P]
lib.conv2d_nhwc_fwd_grouped.restype = _I
lib.conv2d_nhwc_fwd_grouped_pads.argtypes = [_P, _P, _P, _P] + [_I] * 16 + [_P]
lib.conv2d_nhwc_fwd_grouped_pads.restype = _I
lib.conv2d_nhwc_im2col_workspace.argtypes = [_I] * 5
lib.conv2d_nhwc_im2col_workspace.restype = ctypes.c_size_t
lib.conv2d_nhwc_fwd_im2col.argtypes = [_P, _P, _P, _P, ctypes.c_size_t] + [_I] * 6 + [_P]
lib.conv2d_nhwc_fwd_im2col.restype = _I
lib.conv2d_nhwc_fwd_im2col_noalloc.argtypes = [_P, _P, _P] + [_I] * 6 + [_P]
lib.conv2d_nhwc_fwd_im2col_noalloc.restype = _I
lib.dwpw_fwd.argtypes = [_P] * 6 + [_I] * 10 + [_P]
lib.dwpw_fwd.restype = _I
lib.depthwise_fwd.argtypes = [_P, _P, _P, _P] + [_I] * 11 + [_P]
lib.depthwise_fwd.restype = _I
_F = ctypes.c_float
lib.conv_i8_row_pitch.argtypes = [_I]
lib.conv_i8_row_pitch.restype = _I
lib.rmsnorm_i8_fwd.argtypes = [_P] * 6 + [_I] * 3 + [_F, _I, _P]
lib.rmsnorm_i8_fwd.restype = _I
lib.quant_rows_i8_fwd.argtypes = [_P] * 3 + [_I] * 5 + [_P]
lib.quant_rows_i8_fwd.restype = _I
lib.quant_filter_i8_fwd.argtypes = [_P] * 3 + [_I] * 4 + [_P]
lib.quant_filter_i8_fwd.restype = _I
lib.dequant_rows_i8_fwd.argtypes = [_P] * 3 + [_I] * 4 + [_P]
lib.dequant_rows_i8_fwd.restype = _I
lib.pointwise_i8_fwd.argtypes = [_P] * 6 + [_I] * 6 + [_P]
lib.pointwise_i8_fwd.restype = _I
lib.conv2d_nhwc_i8_workspace.argtypes = [_I] * 4
lib.conv2d_nhwc_i8_workspace.restype = ctypes.c_size_t
lib.conv2d_nhwc_fwd_i8.argtypes = [_P, _P, _F] + [_P] * 5 + [ctypes.c_size_t] + [_I] * 6 + [_P]
lib.conv2d_nhwc_fwd_i8.restype = _I
lib.conv_status_string.argtypes = [_I]
lib.conv_status_string.restype = ctypes.c_char_p
lib.conv_device_status.argtypes = [_P, _I]
lib.conv_device_status.restype = _I
lib.conv_last_kernel.argtypes = []
lib.conv_last_kernel.restype = ctypes.c_char_p
lib.conv_selftest_wait_timeout.argtypes = [_P]
lib.conv_selftest_wait_timeout.restype = _I
lib.conv_debug_bounds_build.argtypes = []
lib.conv_debug_bounds_build.restype = _I
lib.conv_debug_bounds_info.argtypes = [ctypes.POINTER(ctypes.c_longlong), _I]
lib.conv_debug_bounds_info.restype = _I
lib.conv_selftest_bounds.argtypes = [_P]
lib.conv_selftest_bounds.restype = _I

EXPORTS = ("conv2d_nhwc_fwd", "conv2d_nhwc_fwd_f32", "conv2d_nhwc_fwd_ex", "conv2d_nhwc_fwd_grouped",
           "conv2d_nhwc_fwd_grouped_pads",
           "conv2d_nhwc_im2col_workspace", "conv2d_nhwc_fwd_im2col", "conv2d_nhwc_fwd_im2col_noalloc", "dwpw_fwd",
           "depthwise_fwd", "conv_status_string", "conv_device_status", "conv_last_kernel",
           "conv_selftest_wait_timeout", "conv_debug_bounds_build", "conv_debug_bounds_info",
           "conv_selftest_bounds", "conv_i8_row_pitch", "rmsnorm_i8_fwd", "quant_rows_i8_fwd", "quant_filter_i8_fwd",
           "dequant_rows_i8_fwd", "pointwise_i8_fwd", "conv2d_nhwc_i8_workspace", "conv2d_nhwc_fwd_i8")
CONV_IM2COL_STATIC_BYTES = 32 * 1024 * 1024   # the scratch of conv2d_nhwc_fwd_im2col_noalloc


class ConvError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {conv_status_string(code)} ({code})")
        self.code = code


def conv_status_string(code: int) -> str:
    return lib.conv_status_string(int(code)).decode()


def _check(code: int, what: str) -> None:
    if code != CONV_OK:
        raise ConvError(code, what)


def _stream(stream, device):
    """The stream handle for a call on `device` (its current stream when None)."""
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    if isinstance(stream, torch.cuda.Stream) and stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _device(*tensors):
    """The one CUDA device every given tensor (None skipped) lives on."""
    devs = {t.device for t in tensors if t is not None}
    if len(devs) != 1:
        raise ValueError(f"all tensors must be on one CUDA device, got {sorted(map(str, devs))}")
    return devs.pop()


def _empty_on(stream, shape, dtype, device):
    """Uninitialised memory that a call on `stream` (the device's current one when None) uses: from the
    allocator's blocks of that stream, as under torch.cuda.stream(stream). A block of another stream
    could still be in use there when this call writes it, and a workspace dropped at return could
    be handed out there while this call's kernels run."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    handle = _stream(stream, device).value or 0
    if not isinstance(stream, torch.cuda.Stream):   # a handle; 0 and 1 are the default stream
        stream = torch.cuda.ExternalStream(handle, device=device) if handle > 1 else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _call(fn, what, tensors, stream, *args):
    """Runs one C entry point with the tensors' device current (the library launches on the
    current device) and its stream as the last argument."""
    import torch
    dev = _device(*tensors)
    with torch.cuda.device(dev):
        _check(fn(*args, _stream(stream, dev)), what)


def _tensor(t, dtype, ndim, name):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {t.dim()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (the C ABI takes dense row-major tensors); "
                         "call .contiguous() first")
    return ctypes.c_void_p(t.data_ptr())


def _dense(X, F, Y, stream, dtype, fn, what):
    import torch
    px = _tensor(X, dtype, 4, "X")
    pf = _tensor(F, dtype, 4, "F")
    N, H, W, Cin = X.shape
    K, K2, Cin2, Cout = F.shape
    if K != K2 or Cin2 != Cin:
        raise ValueError("F must be [K, K, Cin, Cout] matching X")
    if K > min(H, W):
        raise ValueError("K must not exceed min(H, W)")
    if Y is None:
        Y = _empty_on(stream, (N, H - K + 1, W - K + 1, Cout), dtype, X.device)
    elif tuple(Y.shape) != (N, H - K + 1, W - K + 1, Cout):
        raise ValueError("Y has the wrong shape")
    py = _tensor(Y, dtype, 4, "Y")
    _call(fn, what, (X, F, Y), stream, px, pf, py, N, H, W, Cin, Cout, K)
    return Y


def conv2d_nhwc_fwd(X, F, Y=None, stream=None):
    """Dense NHWC convolution, bfloat16: X [N,H,W,Cin], F [K,K,Cin,Cout] -> Y [N,Ho,Wo,Cout]."""
    import torch
    return _dense(X, F, Y, stream, torch.bfloat16, lib.conv2d_nhwc_fwd, "conv2d_nhwc_fwd")


def conv2d_nhwc_fwd_f32(X, F, Y=None, stream=None):
    """Dense NHWC convolution, float32 tensors."""
    import torch
    return _dense(X, F, Y, stream, torch.float32, lib.conv2d_nhwc_fwd_f32, "conv2d_nhwc_fwd_f32")


def conv2d_nhwc_fwd_ex(X, F, bias=None, Y=None, stride=1, pad=0, dil=1, stream=None):
    """Dense NHWC convolution, bfloat16, with stride, zero padding, dilation and an optional
    float32 bias [Cout]: X [N,H,W,Cin], F [K,K,Cin,Cout] -> Y [N,Ho,Wo,Cout]."""
    import torch
    px = _tensor(X, torch.bfloat16, 4, "X")
    pf = _tensor(F, torch.bfloat16, 4, "F")
    N, H, W, Cin = X.shape
    K, K2, Cin2, Cout = F.shape
    if K != K2 or Cin2 != Cin:
        raise ValueError("F must be [K, K, Cin, Cout] matching X")
    pb = ctypes.c_void_p(None)
    if bias is not None:
        pb = _tensor(bias, torch.float32, 1, "bias")
        if bias.shape[0] != Cout:
            raise ValueError("bias must have Cout entries")
    Ho = (H + 2 * pad - (dil * (K - 1) + 1)) // stride + 1
    Wo = (W + 2 * pad - (dil * (K - 1) + 1)) // stride + 1
    if Ho < 1 or Wo < 1:
        raise ValueError("empty output")
    if Y is None:
        Y = _empty_on(stream, (N, Ho, Wo, Cout), torch.bfloat16, X.device)
    elif tuple(Y.shape) != (N, Ho, Wo, Cout):
        raise ValueError("Y has the wrong shape")
    py = _tensor(Y, torch.bfloat16, 4, "Y")
    _call(lib.conv2d_nhwc_fwd_ex, "conv2d_nhwc_fwd_ex", (X, F, bias, Y), stream,
          px, pf, pb, py, N, H, W, Cin, Cout, K, stride, pad, dil)
    return Y


def _pair(v, name):
    if isinstance(v, (tuple, list)):
        if len(v) != 2:
            raise ValueError(f"{name} must be an int or a pair")
        return int(v[0]), int(v[1])
    return int(v), int(v)


def _pads(pad):
    """(top, bottom, left, right) from one int, an (h, w) pair, or ((top, bottom), (left, right))."""
    if isinstance(pad, (tuple, list)):
        if len(pad) != 2:
            raise ValueError("pad must be an int, an (h, w) pair or ((top, bottom), (left, right))")
        out = []
        for v in pad:
            if isinstance(v, (tuple, list)):
                if len(v) != 2:
                    raise ValueError("a per-axis pad must be an int or a (before, after) pair")
                out += [int(v[0]), int(v[1])]
            else:
                out += [int(v), int(v)]
        return tuple(out)
    return (int(pad),) * 4


def conv2d_nhwc_fwd_grouped(X, F, bias=None, Y=None, stride=1, pad=0, dil=1, groups=1, stream=None):
    """Grouped dense NHWC convolution, bfloat16, with a KH x KW filter, per-axis stride and
    dilation (ints or (h, w) pairs), zero padding (an int, an (h, w) pair, or ((top, bottom),
    (left, right)) for different padding before and after an axis -- a causal Conv1D is
    pad=(0, (KW-1, 0))) and an optional float32 bias [Cout]:
    X [N,H,W,Cin], F [KH,KW,Cin/groups,Cout] -> Y [N,Ho,Wo,Cout]. A Conv1D is H = KH = 1."""
    import torch
    px = _tensor(X, torch.bfloat16, 4, "X")
    pf = _tensor(F, torch.bfloat16, 4, "F")
    N, H, W, Cin = X.shape
    KH, KW, Cg, Cout = F.shape
    groups = int(groups)
    if groups < 1 or Cin % groups or Cout % groups or Cg != Cin // groups:
        raise ValueError("F must be [KH, KW, Cin/groups, Cout] with groups dividing Cin and Cout")
    (sh, sw), (dh, dw) = _pair(stride, "stride"), _pair(dil, "dil")
    pt, pb, pl, pr = _pads(pad)
    pbias = ctypes.c_void_p(None)
    if bias is not None:
        pbias = _tensor(bias, torch.float32, 1, "bias")
        if bias.shape[0] != Cout:
            raise ValueError("bias must have Cout entries")
    Ho = (H + pt + pb - (dh * (KH - 1) + 1)) // sh + 1
    Wo = (W + pl + pr - (dw * (KW - 1) + 1)) // sw + 1
    if Ho < 1 or Wo < 1:
        raise ValueError("empty output")
    if Y is None:
        Y = _empty_on(stream, (N, Ho, Wo, Cout), torch.bfloat16, X.device)
    elif tuple(Y.shape) != (N, Ho, Wo, Cout):
        raise ValueError("Y has the wrong shape")
    py = _tensor(Y, torch.bfloat16, 4, "Y")
    if pt == pb and pl == pr:
        _call(lib.conv2d_nhwc_fwd_grouped, "conv2d_nhwc_fwd_grouped", (X, F, bias, Y), stream,
              px, pf, pbias, py, N, H, W, Cin, Cout, KH, KW, sh, sw, pt, pl, dh, dw, groups)
    else:
        _call(lib.conv2d_nhwc_fwd_grouped_pads, "conv2d_nhwc_fwd_grouped_pads", (X, F, bias, Y), stream,
              px, pf, pbias, py, N, H, W, Cin, Cout, KH, KW, sh, sw, pt, pb, pl, pr, dh, dw, groups)
    return Y


def conv2d_nhwc_fwd_im2col(X, F, Y=None, workspace=None, stream=None):
    """Comparison path: explicit patch matrix in `workspace` (allocated here if None, as a uint8
    CUDA tensor of conv2d_nhwc_im2col_workspace bytes), then one cuBLAS GEMM."""
    import torch
    px = _tensor(X, torch.bfloat16, 4, "X")
    pf = _tensor(F, torch.bfloat16, 4, "F")
    N, H, W, Cin = X.shape
    K, K2, Cin2, Cout = F.shape
    if K != K2 or Cin2 != Cin:
        raise ValueError("F must be [K, K, Cin, Cout] matching X")
    need = lib.conv2d_nhwc_im2col_workspace(N, H, W, Cin, K)
    if need == 0:
        raise ValueError("invalid shape")
    if workspace is None:
        workspace = _empty_on(stream, need, torch.uint8, X.device)
    if not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    if Y is None:
        Y = _empty_on(stream, (N, H - K + 1, W - K + 1, Cout), torch.bfloat16, X.device)
    elif tuple(Y.shape) != (N, H - K + 1, W - K + 1, Cout):
        raise ValueError("Y has the wrong shape")
    py = _tensor(Y, torch.bfloat16, 4, "Y")
    _call(lib.conv2d_nhwc_fwd_im2col, "conv2d_nhwc_fwd_im2col", (X, F, Y, workspace), stream,
          px, pf, py, ctypes.c_void_p(workspace.data_ptr()), workspace.numel() * workspace.element_size(),
          N, H, W, Cin, Cout, K)
    return Y


def conv2d_nhwc_fwd_im2col_noalloc(X, F, Y, stream=None):
    """The explicit-im2col comparison path with its patch matrix in the library's static scratch
    (CONV_IM2COL_STATIC_BYTES per device) instead of a workspace, for callers that cannot
    allocate device memory. Y must be passed: this binding allocates nothing either."""
    import torch
    px = _tensor(X, torch.bfloat16, 4, "X")
    pf = _tensor(F, torch.bfloat16, 4, "F")
    N, H, W, Cin = X.shape
    K, K2, Cin2, Cout = F.shape
    if K != K2 or Cin2 != Cin:
        raise ValueError("F must be [K, K, Cin, Cout] matching X")
    if K > min(H, W):
        raise ValueError("K must not exceed min(H, W)")
    if tuple(Y.shape) != (N, H - K + 1, W - K + 1, Cout):
        raise ValueError("Y has the wrong shape")
    py = _tensor(Y, torch.bfloat16, 4, "Y")
    _call(lib.conv2d_nhwc_fwd_im2col_noalloc, "conv2d_nhwc_fwd_im2col_noalloc", (X, F, Y), stream,
          px, pf, py, N, H, W, Cin, Cout, K)
    return Y


def depthwise_fwd(x, w, bias=None, y=None, stride=1, pad=0, dil=1, mode=DW_EXACT, stream=None):
    """Depthwise convolution, float32: x [N,Cin,H,W], w [Cin*mult,KH,KW], bias [Cin*mult] or None."""
    import torch
    px = _tensor(x, torch.float32, 4, "x")
    pw = _tensor(w, torch.float32, 3, "w")
    N, Cin, H, W = x.shape
    Cout, KH, KW = w.shape
    if Cout % Cin != 0:
        raise ValueError("w must have Cin * mult planes")
    mult = Cout // Cin
    pb = ctypes.c_void_p(None)
    if bias is not None:
        pb = _tensor(bias, torch.float32, 1, "bias")
        if bias.shape[0] != Cout:
            raise ValueError("bias must have Cin * mult entries")
    Ho = (H + 2 * pad - (dil * (KH - 1) + 1)) // stride + 1
    Wo = (W + 2 * pad - (dil * (KW - 1) + 1)) // stride + 1
    if Ho < 1 or Wo < 1:
        raise ValueError("empty output")
    if y is None:
        y = _empty_on(stream, (N, Cout, Ho, Wo), torch.float32, x.device)
    elif tuple(y.shape) != (N, Cout, Ho, Wo):
        raise ValueError("y has the wrong shape")
    py = _tensor(y, torch.float32, 4, "y")
    _call(lib.depthwise_fwd, "depthwise_fwd", (x, w, bias, y), stream,
          px, pw, pb, py, N, Cin, mult, H, W, KH, KW, stride, pad, dil, int(mode))
    return y


def dwpw_fwd(x, w_dw, b_dw, F, b_pw=None, y=None, stride=1, pad=0, dil=1, mode=DW_EXACT, stream=None):
    """Depthwise then pointwise, fused: x float32 [N,C,H,W], w_dw float32 [C,K,K], b_dw float32
    [C] or None, F bfloat16 [C,Cout], b_pw float32 [Cout] or None -> y float32 [N,Cout,Ho,Wo]."""
    import torch
    px = _tensor(x, torch.float32, 4, "x")
    pw = _tensor(w_dw, torch.float32, 3, "w_dw")
    pf = _tensor(F, torch.bfloat16, 2, "F")
    N, C, H, W = x.shape
    C2, K, K2 = w_dw.shape
    if C2 != C or K != K2:
        raise ValueError("w_dw must be [C, K, K]")
    C3, Cout = F.shape
    if C3 != C:
        raise ValueError("F must be [C, Cout]")
    pbd = ctypes.c_void_p(None)
    if b_dw is not None:
        pbd = _tensor(b_dw, torch.float32, 1, "b_dw")
        if b_dw.shape[0] != C:
            raise ValueError("b_dw must have C entries")
    pbp = ctypes.c_void_p(None)
    if b_pw is not None:
        pbp = _tensor(b_pw, torch.float32, 1, "b_pw")
        if b_pw.shape[0] != Cout:
            raise ValueError("b_pw must have Cout entries")
    Ho = (H + 2 * pad - (dil * (K - 1) + 1)) // stride + 1
    Wo = (W + 2 * pad - (dil * (K - 1) + 1)) // stride + 1
    if Ho < 1 or Wo < 1:
        raise ValueError("empty output")
    if y is None:
        y = _empty_on(stream, (N, Cout, Ho, Wo), torch.float32, x.device)
    elif tuple(y.shape) != (N, Cout, Ho, Wo):
        raise ValueError("y has the wrong shape")
    py = _tensor(y, torch.float32, 4, "y")
    _call(lib.dwpw_fwd, "dwpw_fwd", (x, w_dw, b_dw, F, b_pw, y), stream,
          px, pw, pbd, pf, pbp, py, N, C, H, W, K, stride, pad, dil, Cout, int(mode))
    return y


# ---- 8-bit operators ---------------------------------------------------------------------
# A single-token call of these takes 2 to 5 us on the GPU, so the host's part counts. On the current
# stream a call goes through _binding_i8 (csrc/binding_i8.cpp), which looks at the tensors in C++: 3
# to 5 us with the outputs given. What it does not find in order, and a call with a stream named,
# takes the checked way below, which says what is wrong. The checked way needs no extension: where
# none can be built or loaded (no compiler), every call takes it, after a warning.
_BF16 = _F32 = _INT8 = _empty = _Tensor = _fast = None
_ASK_SLOW = -1000


class _NoShortPath:
    """In the extension's place where there is none: every call asks for the checked way."""

    @staticmethod
    def _ask(*args):
        return _ASK_SLOW

    rmsnorm = rows = filter = dequant = pointwise = layer = _ask


def _i8_extension():
    import importlib.util
    spec = importlib.util.spec_from_file_location("_binding_i8", _build.build_binding())
    fast = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(fast)
    fast.bind(*(ctypes.cast(f, _P).value for f in (lib.rmsnorm_i8_fwd, lib.quant_rows_i8_fwd, lib.quant_filter_i8_fwd,
                                                   lib.dequant_rows_i8_fwd, lib.pointwise_i8_fwd, lib.conv2d_nhwc_fwd_i8)))
    return fast


def _i8_init():
    global _BF16, _F32, _INT8, _empty, _Tensor, _fast
    import torch
    _BF16, _F32, _INT8, _empty, _Tensor = torch.bfloat16, torch.float32, torch.int8, torch.empty, torch.Tensor
    try:
        fast = _i8_extension()
    except (RuntimeError, OSError, ImportError) as e:
        import warnings
        warnings.warn(f"the 8-bit operators run without their short host path: {e}", RuntimeWarning, stacklevel=3)
        fast = _NoShortPath()
    _fast = fast
    return fast


def _i8_is_matrix(t):
    """Whether outputs can be shaped after t; otherwise the checked way says why not."""
    if _fast is None:
        _i8_init()
    return isinstance(t, _Tensor) and t.ndim == 2 and t.is_cuda and t.numel() > 0


def _i8_quick(rc, what):
    """Whether the short path made the call; its error raised."""
    if rc == CONV_OK:
        return True
    if rc != _ASK_SLOW:
        _check(rc, what)
    return False


def _i8_sizes(name, *sizes):
    """The C ABI's sizes are int: larger ones must not be cut to their low bits on the way."""
    if max(sizes) > 2 ** 31 - 1:
        raise ValueError(f"{name} is larger than 2^31 - 1 in a dimension")


def _i8_matrix(x, name):
    """(conv_dtype, address) of a contiguous bfloat16 or float32 CUDA matrix."""
    import torch
    if _fast is None:
        _i8_init()
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dtype is not _BF16 and x.dtype is not _F32:
        raise TypeError(f"{name} must be torch.bfloat16 or torch.float32, got {x.dtype}")
    _tensor(x, x.dtype, 2, name)
    _i8_sizes(name, *x.shape)
    return CONV_BF16 if x.dtype is _BF16 else CONV_F32, x.data_ptr()


def _i8_ptr(t, dtype, shape, name):
    """The address of a contiguous CUDA tensor of the given type and shape."""
    p = _tensor(t, dtype, len(shape), name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return p


def _i8_rows(t, name):
    """(address, rows, columns, row pitch) of an int8 matrix whose rows start on 16-byte boundaries."""
    import torch
    if _fast is None:
        _i8_init()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not _INT8:
        raise TypeError(f"{name} must be torch.int8, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dimensions, got {t.dim()}")
    n, c = t.shape
    pitch, step = t.stride()
    if n < 2:
        pitch = (c + 15) // 16 * 16   # the stride of a dimension with one element means nothing
    _i8_sizes(name, n, c, pitch)
    if (step != 1 and c > 1) or pitch < c or pitch % 16:
        raise ValueError(f"{name} must be an int8 matrix whose rows are contiguous and start on 16-byte boundaries "
                         "(empty_rows_i8 makes one)")
    return t.data_ptr(), n, c, pitch


def empty_rows_i8(rows, C, device="cuda"):
    """An uninitialised int8 matrix [rows, C] in the layout the 8-bit operators take, a view of
    [rows, pitch] whose rows start where conv_i8_row_pitch puts them. Copy 8-bit rows from
    elsewhere (a checkpoint's filter) into one with copy_()."""
    return _i8_empty_rows(rows, C, device, None)


def _i8_empty_rows(rows, C, device, stream):
    import torch
    _i8_sizes("the matrix", int(rows), int(C))
    pitch = lib.conv_i8_row_pitch(int(C))
    if pitch == 0 or rows < 1:
        raise ValueError("rows and C must be positive")
    return _empty_on(stream, (rows, pitch), torch.int8, device)[:, :C]


def _i8_out(q, scale, rows, C, device, stream):
    """q and scale (allocated where None), their addresses and q's pitch."""
    if q is None:
        q = _i8_empty_rows(rows, C, device, stream)
    if scale is None:
        scale = _empty_on(stream, rows, _F32, device)
    pq, n, c, pitch = _i8_rows(q, "q")
    if n != rows or c != C:
        raise ValueError(f"q must have shape {(rows, C)}, got {(n, c)}")
    return q, scale, pq, pitch, _i8_ptr(scale, _F32, (rows,), "scale")


def _i8_result(y, dtype, shape, device, stream):
    """y (allocated where None), its conv_dtype and its address."""
    if y is None:
        y = _empty_on(stream, shape, _BF16 if dtype is None else dtype, device)
    elif dtype is not None and y.dtype is not dtype:
        raise TypeError(f"y must be {dtype}, got {y.dtype}")
    if y.dtype is _BF16:
        return y, CONV_BF16, _i8_ptr(y, _BF16, shape, "y")
    if y.dtype is _F32:
        return y, CONV_F32, _i8_ptr(y, _F32, shape, "y")
    raise TypeError(f"y must be torch.bfloat16 or torch.float32, got {y.dtype}")


def rmsnorm_i8_fwd(x, weight, residual=None, h=None, q=None, scale=None, eps=1e-6, stream=None):
    """Root-mean-square norm of the rows of x [M, C] (bfloat16 or float32), with a residual's
    addition before it, and 8-bit rows out: h = x + residual (rounded to x's type; x itself without
    a residual), then h * weight / sqrt(mean(h^2) + eps) as int8 q [M, C] and float32 scale [M].
    weight is float32 [C]. h may be x or residual (updated in place). Returns (q, scale, h); h is
    None without a residual."""
    if stream is None:
        oq, os, oh = q, scale, h
        if (oq is None or os is None or (oh is None and residual is not None)) and _i8_is_matrix(x):
            oq = empty_rows_i8(*x.shape, x.device) if oq is None else oq
            os = _empty(x.shape[0], dtype=_F32, device=x.device) if os is None else os
            oh = _empty(x.shape, dtype=x.dtype, device=x.device) if oh is None and residual is not None else oh
        if _i8_quick((_fast or _i8_init()).rmsnorm(x, weight, residual, oh, oq, os, eps), "rmsnorm_i8_fwd"):
            return oq, os, oh
    dt, px = _i8_matrix(x, "x")
    shape = x.shape
    M, C = shape
    pw = _i8_ptr(weight, _F32, (C,), "weight")
    pr = ph = None
    if residual is not None:
        pr = _i8_ptr(residual, x.dtype, shape, "residual")
        if h is None:
            h = _empty_on(stream, shape, x.dtype, x.device)
        ph = _i8_ptr(h, x.dtype, shape, "h")
    elif h is not None:
        raise ValueError("h is x + residual: give the residual too")
    q, scale, pq, ldq, ps = _i8_out(q, scale, M, C, x.device, stream)
    _call(lib.rmsnorm_i8_fwd, "rmsnorm_i8_fwd", (residual, weight, h, q, scale, x), stream,
             px, pr, pw, ph, pq, ps, M, C, ldq, float(eps), dt)
    return q, scale, h


def quant_rows_i8_fwd(x, glu=False, q=None, scale=None, stream=None):
    """8-bit rows of x [M, C] (bfloat16 or float32): int8 q [M, C] and float32 scale [M], one per row.
    With glu, x is [M, 2C] and the rows are silu(x[:, :C]) * x[:, C:]. Returns (q, scale)."""
    if stream is None:
        oq, os = q, scale
        if (oq is None or os is None) and _i8_is_matrix(x):
            C = x.shape[1]
            oq = empty_rows_i8(x.shape[0], (C // 2 or 1) if glu else C, x.device) if oq is None else oq
            os = _empty(x.shape[0], dtype=_F32, device=x.device) if os is None else os
        if _i8_quick((_fast or _i8_init()).rows(x, oq, os, True if glu else False), "quant_rows_i8_fwd"):
            return oq, os
    dt, px = _i8_matrix(x, "x")
    M, C = x.shape
    if glu:
        if C % 2:
            raise ValueError("glu needs x [M, 2C]")
        C //= 2
    q, scale, pq, ldq, ps = _i8_out(q, scale, M, C, x.device, stream)
    _call(lib.quant_rows_i8_fwd, "quant_rows_i8_fwd", (q, scale, x), stream,
             px, pq, ps, M, C, ldq, 1 if glu else 0, dt)
    return q, scale


def quant_filter_i8_fwd(F, q=None, scale=None, stream=None):
    """8-bit rows of a 1 x 1 filter F [Cin, Cout] or [1, 1, Cin, Cout] (bfloat16 or float32): int8
    q [Cout, Cin], transposed, and float32 scale [Cout], one per output channel. Returns (q, scale)."""
    if getattr(F, "ndim", 0) == 4:
        if tuple(F.shape[:2]) != (1, 1):
            raise ValueError("F must be a 1 x 1 filter")
        F = F[0, 0]
    if stream is None:
        oq, os = q, scale
        if (oq is None or os is None) and _i8_is_matrix(F):
            oq = empty_rows_i8(F.shape[1], F.shape[0], F.device) if oq is None else oq
            os = _empty(F.shape[1], dtype=_F32, device=F.device) if os is None else os
        if _i8_quick((_fast or _i8_init()).filter(F, oq, os), "quant_filter_i8_fwd"):
            return oq, os
    dt, pf = _i8_matrix(F, "F")
    Cin, Cout = F.shape
    q, scale, pq, ldw, ps = _i8_out(q, scale, Cout, Cin, F.device, stream)
    _call(lib.quant_filter_i8_fwd, "quant_filter_i8_fwd", (q, scale, F), stream,
             pf, pq, ps, Cin, Cout, ldw, dt)
    return q, scale


def dequant_rows_i8_fwd(q, scale, y=None, dtype=None, stream=None):
    """Reads 8-bit rows back: y [M, C] = q * scale, in y's type (dtype, bfloat16 by default)."""
    if stream is None and (y is None or dtype is None):
        out = y
        if y is None and _i8_is_matrix(q):
            out = _empty(q.shape, dtype=dtype or _BF16, device=q.device)
        if _i8_quick((_fast or _i8_init()).dequant(q, scale, out), "dequant_rows_i8_fwd"):
            return out
    pq, M, C, ldq = _i8_rows(q, "q")
    ps = _i8_ptr(scale, _F32, (M,), "scale")
    y, dt, py = _i8_result(y, dtype, (M, C), q.device, stream)
    _call(lib.dequant_rows_i8_fwd, "dequant_rows_i8_fwd", (scale, y, q), stream,
             pq, ps, py, M, C, ldq, dt)
    return y


def pointwise_i8_fwd(q, q_scale, Wq, w_scale, bias=None, y=None, dtype=None, stream=None):
    """The product of 8-bit rows: y [M, Cout] = (q [M, Cin] @ Wq [Cout, Cin]^T) * q_scale [M] * w_scale [Cout]
    + bias [Cout], the sum exact in int32, in y's type (dtype, bfloat16 by default)."""
    if stream is None and (y is None or dtype is None):
        out = y
        if y is None and _i8_is_matrix(q) and _i8_is_matrix(Wq):
            out = _empty((q.shape[0], Wq.shape[0]), dtype=dtype or _BF16, device=q.device)
        if _i8_quick((_fast or _i8_init()).pointwise(q, q_scale, Wq, w_scale, bias, out), "pointwise_i8_fwd"):
            return out
    pq, M, Cin, ldq = _i8_rows(q, "q")
    pw, Cout, Cin2, ldw = _i8_rows(Wq, "Wq")
    if Cin2 != Cin:
        raise ValueError(f"Wq must have q's {Cin} columns, got {Cin2}")
    ps, pws = _i8_ptr(q_scale, _F32, (M,), "q_scale"), _i8_ptr(w_scale, _F32, (Cout,), "w_scale")
    pb = None if bias is None else _i8_ptr(bias, _F32, (Cout,), "bias")
    y, dt, py = _i8_result(y, dtype, (M, Cout), q.device, stream)
    _call(lib.pointwise_i8_fwd, "pointwise_i8_fwd", (q_scale, Wq, w_scale, bias, y, q), stream,
             pq, ps, pw, pws, pb, py, M, Cin, Cout, ldq, ldw, dt)
    return y


def conv2d_nhwc_fwd_i8(X, Wq, w_scale, bias=None, norm=None, eps=1e-6, Y=None, workspace=None, stream=None):
    """Dense NHWC 1 x 1 convolution in 8-bit integers: X bfloat16 [N,H,W,Cin], quantised per pixel
    (with norm, float32 [Cin]: after a root-mean-square norm with that weight), times the filter Wq
    int8 [Cout, Cin] with w_scale [Cout] (quant_filter_i8_fwd) -> Y bfloat16 [N,H,W,Cout].
    workspace: a uint8 CUDA tensor of at least conv2d_nhwc_i8_workspace bytes, allocated here if None."""
    if stream is None and Y is not None and workspace is not None and \
            _i8_quick((_fast or _i8_init()).layer(X, norm, eps, Wq, w_scale, bias, Y, workspace), "conv2d_nhwc_fwd_i8"):
        return Y
    import torch
    pw, Cout, Cin2, ldw = _i8_rows(Wq, "Wq")
    px = _tensor(X, torch.bfloat16, 4, "X")
    N, H, W, Cin = X.shape
    _i8_sizes("X", N, H, W, Cin)
    if Cin2 != Cin:
        raise ValueError(f"Wq must have X's {Cin} channels, got {Cin2}")
    pws = _i8_ptr(w_scale, _F32, (Cout,), "w_scale")
    pb = None if bias is None else _i8_ptr(bias, _F32, (Cout,), "bias")
    pn = None if norm is None else _i8_ptr(norm, _F32, (Cin,), "norm")
    if workspace is None:
        need = lib.conv2d_nhwc_i8_workspace(N, H, W, Cin)
        if need == 0:
            raise ValueError("invalid shape")
        workspace = _empty_on(stream, need, torch.uint8, X.device)
    elif not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    if Y is None:
        Y = _empty_on(stream, (N, H, W, Cout), torch.bfloat16, X.device)
    py = _i8_ptr(Y, _BF16, (N, H, W, Cout), "Y")
    _call(lib.conv2d_nhwc_fwd_i8, "conv2d_nhwc_fwd_i8", (norm, Wq, w_scale, bias, Y, workspace, X), stream,
             px, pn, float(eps), pw, pws, pb, py, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
             N, H, W, Cin, Cout, ldw)
    return Y


def conv_last_kernel() -> str:
    """Kernel family the last successful call on this thread launched (the dispatcher's choice)."""
    return lib.conv_last_kernel().decode()


def _current():
    import torch
    return torch.device("cuda", torch.cuda.current_device())


def conv_selftest_wait_timeout(stream=None) -> int:
    """Runs the bounded-wait diagnostic (about one second) on the current device; returns the
    launch status."""
    return lib.conv_selftest_wait_timeout(_stream(stream, _current()))


def conv_selftest_bounds(stream=None) -> int:
    """Runs the bounds-check diagnostic (a failing check that touches no memory) on the current
    device; returns the launch status."""
    return lib.conv_selftest_bounds(_stream(stream, _current()))


def conv_debug_bounds_build() -> bool:
    """True when the loaded library is the bounds-checked build."""
    return lib.conv_debug_bounds_build() == 1


def conv_debug_bounds_info(reset=False):
    """First failed bounds check on the current device since the last reset, as (site, index,
    limit), or None; always None in the normal build."""
    info = (ctypes.c_longlong * 3)()
    rc = lib.conv_debug_bounds_info(info, 1 if reset else 0)
    if rc != CONV_OK:
        raise ConvError(rc, "conv_debug_bounds_info")
    return None if info[0] < 0 else (info[0], info[1], info[2])


def conv_device_status(stream=None, reset=False) -> int:
    """Synchronises the stream and returns the current device's status word as a conv_status
    code."""
    return lib.conv_device_status(_stream(stream, _current()), 1 if reset else 0)
