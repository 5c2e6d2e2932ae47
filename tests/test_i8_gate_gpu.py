"""The gate of quant_rows_i8_fwd at the error bound that its documentation gives."""
import os
import re

import pytest
import torch

from tests.conftest import ROOT

U = 2.0 ** -24   # half a step of float32


def _bound(text):
    """(constant, factor of |a|) of the documented bound, in units of 2^-24."""
    m = re.search(r"relative error below\s+(?:\*\s+)?\((\d+) \+ ([\d.]+) \|(?:a|x\[c\])\|\) 2\^-24", text)
    assert m, "the bound's sentence"
    return float(m.group(1)), float(m.group(2))


def documented_bound():
    with open(os.path.join(ROOT, "include", "conv_b200.h")) as f:
        return _bound(f.read())


def test_the_header_and_the_kernel_state_one_bound():
    with open(os.path.join(ROOT, "cnn_convolution_nhwc_b200", "csrc", "i8_rows.cuh")) as f:
        assert _bound(f.read()) == documented_bound()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lo,hi", [(-87.3, -60), (-60, -20), (-20, -1), (-1, 1), (1, 20), (20, 88)])
def test_gate_error(cuda, lo, hi, dtype):
    # rows of one value: the scale is |silu(a) * up| / 127, rounded once more
    import cnn_convolution_nhwc_b200 as cb
    c0, c1 = documented_bound()
    g = torch.Generator("cuda").manual_seed(17)
    n = 1 << 20
    a = (torch.rand(n, generator=g, device="cuda") * (hi - lo) + lo).clamp(-87.3, 88).to(dtype)
    a = torch.where(a < -87.32, torch.full_like(a, -87.0), a)
    for up in (torch.ones_like(a), torch.randn(n, generator=g, device="cuda").to(dtype)):
        q, s = cb.quant_rows_i8_fwd(torch.stack([a, up], dim=1), glu=True)
        gate = a.double()
        v = gate / (1 + torch.exp(-gate)) * up.double()
        v[gate < -87.33] = 0   # as documented; -87.5 is among the bf16 gates
        # the scale's rounding: half a step, at least of the smallest denormal
        off = ((c0 + c1 * gate.abs()) * U + U) * v.abs() + 127 * 2.0 ** -150 * (1 + 1 / 127) + 2.0 ** -150
        assert bool(((s.double() * 127 - v.abs()).abs() <= off).all())
        assert bool((q[:, 0].double().sign() == v.sign())[v.abs() > 1e-36].all())
