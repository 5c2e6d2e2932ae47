"""The Python extension of the 8-bit operators' short host path: which file is loaded."""
import os
import sysconfig

import pytest
import torch

import cnn_convolution_nhwc_b200 as cb


def test_an_extension_built_for_another_torch_or_python_is_not_loaded(monkeypatch):
    build = cb._build
    here = build.binding_path()
    assert os.path.dirname(here) == build.PKG and here.endswith(".so") and os.path.basename(here).count(os.sep) == 0
    assert build.build_binding() == here and os.path.exists(here)   # built for this torch, at its path
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "2.99.0+cu999")
        other = build.binding_path()
        assert other != here and not os.path.exists(other)
    with monkeypatch.context() as m:
        real = sysconfig.get_config_var
        m.setattr(sysconfig, "get_config_var", lambda name: "cpython-399-x86_64-linux-gnu" if name == "SOABI" else real(name))
        assert build.binding_path() not in (here, other)
    assert build.binding_path() == here


@pytest.mark.parametrize("error", [RuntimeError("g++ failed"), FileNotFoundError("g++"), ImportError("undefined symbol")])
def test_without_an_extension_the_checked_way_is_taken(monkeypatch, error):
    def fail(*a, **k):
        raise error
    monkeypatch.setattr(cb._build, "build_binding", fail)
    monkeypatch.setattr(cb, "_fast", None)
    with pytest.warns(RuntimeWarning, match="short host path"):
        with pytest.raises(ValueError, match="CUDA"):   # the checked way's own refusal of a CPU tensor
            cb.quant_rows_i8_fwd(torch.zeros(2, 8, dtype=torch.bfloat16))
    for call in (lambda: cb.dequant_rows_i8_fwd(torch.zeros(2, 16, dtype=torch.int8), torch.ones(2)),
                 lambda: cb.pointwise_i8_fwd(torch.zeros(2, 16, dtype=torch.int8), torch.ones(2),
                                             torch.zeros(3, 16, dtype=torch.int8), torch.ones(3)),
                 lambda: cb.quant_filter_i8_fwd(torch.zeros(8, 4)),
                 lambda: cb.rmsnorm_i8_fwd(torch.zeros(2, 8), torch.ones(8)),
                 lambda: cb.conv2d_nhwc_fwd_i8(torch.zeros(1, 1, 2, 16, dtype=torch.bfloat16),
                                               torch.zeros(3, 16, dtype=torch.int8), torch.ones(3))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.gpu
def test_the_checked_way_alone_gives_the_same_results(cuda, monkeypatch):
    g = torch.Generator("cuda").manual_seed(3)
    X = torch.randn(1, 5, 7, 96, generator=g, device="cuda").bfloat16()
    F, norm = torch.randn(96, 40, generator=g, device="cuda").bfloat16(), torch.ones(96, device="cuda")
    x = X.reshape(-1, 96)

    def run():
        w, ws = cb.quant_filter_i8_fwd(F)
        q, s, h = cb.rmsnorm_i8_fwd(x, norm, x)
        q2, s2 = cb.quant_rows_i8_fwd(x, glu=True)
        return [w, ws, q, s, h, q2, s2, cb.pointwise_i8_fwd(q, s, w, ws), cb.dequant_rows_i8_fwd(q2, s2),
                cb.conv2d_nhwc_fwd_i8(X, w, ws, norm=norm, Y=torch.empty(1, 5, 7, 40, dtype=torch.bfloat16, device="cuda"))]
    want = run()
    assert not isinstance(cb._fast, cb._NoShortPath)
    monkeypatch.setattr(cb, "_fast", cb._NoShortPath())
    assert all(torch.equal(a, b) for a, b in zip(run(), want))
