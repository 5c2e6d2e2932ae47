"""Outputs that a caller gives with another shape are refused before anything is launched."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cb(cuda):
    import cnn_convolution_nhwc_b200 as m
    return m


def test_given_outputs_of_another_shape(cb):
    X, F = torch.zeros(2, 8, 8, 16, device="cuda").bfloat16(), torch.zeros(3, 3, 16, 16, device="cuda").bfloat16()
    x, w = torch.zeros(1, 4, 8, 8, device="cuda"), torch.zeros(4, 3, 3, device="cuda")
    wq, ws = torch.zeros(16, 16, dtype=torch.int8, device="cuda"), torch.ones(16, device="cuda")
    Y = torch.zeros(2, 6, 5, 16, device="cuda").bfloat16()   # a column of pixels too few
    for call in (lambda: cb.conv2d_nhwc_fwd(X, F, Y=Y), lambda: cb.conv2d_nhwc_fwd_ex(X, F, Y=Y),
                 lambda: cb.conv2d_nhwc_fwd_grouped(X, F, Y=Y), lambda: cb.conv2d_nhwc_fwd_im2col(X, F, Y=Y),
                 lambda: cb.conv2d_nhwc_fwd_im2col_noalloc(X, F, Y),
                 lambda: cb.conv2d_nhwc_fwd_f32(X.float(), F.float(), Y=Y.float()),
                 lambda: cb.depthwise_fwd(x, w, y=torch.zeros(1, 4, 6, 5, device="cuda")),
                 lambda: cb.dwpw_fwd(x, w, None, F[0, 0, :4].contiguous(), y=torch.zeros(1, 16, 6, 5, device="cuda"))):
        with pytest.raises(ValueError, match="wrong shape"):
            call()
    for call in (lambda: cb.conv2d_nhwc_fwd_i8(X, wq, ws, Y=Y),
                 lambda: cb.pointwise_i8_fwd(wq, ws, wq, ws, y=torch.zeros(16, 15, device="cuda")),
                 lambda: cb.dequant_rows_i8_fwd(wq, ws, y=torch.zeros(15, 16, device="cuda"))):
        with pytest.raises(ValueError, match="must have shape"):
            call()
