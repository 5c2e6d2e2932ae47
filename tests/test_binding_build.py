"""The Python extension of the 8-bit operators' short host path: which file is loaded."""
import os
import sysconfig

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
