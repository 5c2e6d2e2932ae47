"""The 8-bit product on every forced plan that fits the shape: the kernel that was asked for runs, agrees with float64,
and agrees bit for bit with every other plan (the sums are integers, and both kernels round alike)."""
import numpy as np
import pytest
import torch

from tests import i8_reference as ref
from tests.test_i8_gpu import U, _bytes, _gen, _normal

pytestmark = pytest.mark.gpu

PLANS = [("pair", 256), ("pair", 128)] + [("split", bn, s) for bn in (16, 32, 64, 128) for s in (1, 2, 4, 8)]
# a reduction of 15 k blocks and more, so that every split fits: odd and even numbers of them, Cin off 128, tokens on both
# sides of the tiles' columns, channels off 128
SHAPES = [(1, 1920, 136), (15, 1801, 300), (16, 2048, 128), (33, 2177, 257), (129, 1900, 1001), (64, 4096, 512), (300, 2300, 264)]


@pytest.fixture(scope="module")
def cb(cuda):
    import cnn_convolution_nhwc_b200 as m
    return m


def fits(plan, Cin):
    return plan[0] == "pair" or plan[2] <= ((Cin + 127) // 128 + 1) // 2


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,Cin,Cout", SHAPES)
def test_every_plan(cb, M, Cin, Cout, dtype, monkeypatch):
    g = _gen(M, Cin, Cout, 7)
    q, wq = _bytes(g, M, Cin, cb, lo=-128), _bytes(g, Cout, Cin, cb, lo=-128)
    qs, ws, bias = _normal(g, M) / 100, _normal(g, Cout) / 100, _normal(g, Cout)
    for b in (None, bias):
        want, mag = ref.product(q, qs, wq, ws, b)
        # as in test_product: four float32 roundings, then the output's
        tol = 4 * U * mag * (1 + ref.round_half(dtype)) + ref.round_half(dtype) * np.abs(want) + 2.0 ** -149
        first = None
        for plan in PLANS:
            assert fits(plan, Cin)
            monkeypatch.setenv("CONV_B200_I8", ",".join(map(str, plan)))
            guard = torch.full((M + 1, Cout), 7.0, dtype=dtype, device="cuda")
            y = cb.pointwise_i8_fwd(q, qs, wq, ws, b, y=guard[:M])
            assert cb.conv_last_kernel() == f"i8_{plan[0]}_kernel", plan
            assert np.all(np.abs(ref.f64(y) - want) <= tol), plan
            assert torch.all(guard[M] == 7.0), plan
            first = y if first is None else first
            assert torch.equal(y, first), plan
    assert cb.conv_device_status() == cb.CONV_OK


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_plans_of_short_reductions(cb, dtype, monkeypatch):
    # one to fourteen k blocks: the splits that still fit, the largest of them with one block of k a CTA
    for kblk in range(1, 15):
        M, Cin, Cout = 20, kblk * 128 - 40, 140
        g = _gen(M, Cin, Cout, 8)
        q, wq = _bytes(g, M, Cin, cb), _bytes(g, Cout, Cin, cb)
        qs, ws = _normal(g, M), _normal(g, Cout)
        first = None
        for plan in PLANS:
            if not fits(plan, Cin):
                continue
            monkeypatch.setenv("CONV_B200_I8", ",".join(map(str, plan)))
            y = cb.pointwise_i8_fwd(q, qs, wq, ws, dtype=dtype)
            assert cb.conv_last_kernel() == f"i8_{plan[0]}_kernel", plan
            if first is None:
                want, mag = ref.product(q, qs, wq, ws, None)
                assert np.all(np.abs(ref.f64(y) - want) <= (4 * U * (1 + ref.round_half(dtype)) + ref.round_half(dtype)) * mag + 2.0 ** -149)
                first = y
            assert torch.equal(y, first), (plan, kblk)
