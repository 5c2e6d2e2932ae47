"""The 8-bit norm at the ends of its range: scales next to the largest float32, and rows so long that the order of
their sum of squares shows."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24   # half a step of float32


@pytest.fixture(scope="module")
def cb(cuda):
    import cnn_convolution_nhwc_b200 as m
    return m


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("C", [64, 77, 520, 4096, 4099, 16400, 16401])
def test_scale_whose_127_fold_passes_the_range(cb, C, dtype):
    # one channel of 1 among zeros: rstd is sqrt(C), and weight * rstd passes 3.4e38 while a 127th of it does not
    x = torch.zeros(2, C, dtype=dtype, device="cuda")
    x[0, C // 2], x[1, C - 1] = 1.0, -1.0
    w = torch.full((C,), 3e38, device="cuda")
    want = float(w[0].double()) * np.sqrt(C / (1 + C * np.float64(np.float32(1e-6)))) / 127
    assert 127 * want > 3.4028235e38 > want
    for residual in (None, torch.zeros_like(x)):
        q, scale, _ = cb.rmsnorm_i8_fwd(x, w, residual, eps=1e-6)
        assert q[0, C // 2] == 127 and q[1, C - 1] == -127 and int(q.int().abs().sum()) == 2 * 127
        # roundings: mean, eps added, root (half of both), quotient, division by 127, product; the sum is exact
        assert np.all(np.abs(scale.double().cpu().numpy() - want) <= 5 * U * want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("value", [1.1, 0.3])
@pytest.mark.parametrize("C", [16384, 28001, 55001, 112001, 1 << 24, (1 << 24) + 5, 1 << 27, (1 << 27) - 3])
def test_sum_of_squares_of_alike_values(cb, C, value, dtype):
    # alike values round alike: the error of a chain of additions grows with its length. The sum is off by
    # less than 2^-17 whatever C; half of that and six roundings (mean, eps, root, quotient, two products) reach the scale
    x = torch.full((1, C), value, dtype=dtype, device="cuda")
    v = float(x[0, 0].double())
    want = v / np.sqrt(v * v + np.float64(np.float32(1e-6))) / 127
    w = torch.ones(C, device="cuda")
    for h in (None, torch.empty_like(x)):
        q, scale, _ = cb.rmsnorm_i8_fwd(x, w, None if h is None else torch.zeros_like(x), h=h, eps=1e-6)
        assert abs(float(scale[0].double()) - want) <= (2.0 ** -18 + 6 * U) * want
        assert bool((q == 127).all())
