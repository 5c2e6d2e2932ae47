"""What every kernel source has to keep for launches that overlap on one stream, checked in the sources."""
import glob
import os
import re

import pytest

from tests.conftest import ROOT

SOURCES = sorted(glob.glob(os.path.join(ROOT, "cnn_convolution_nhwc_b200", "csrc", "*.cu*")))


def _kernels():
    """(file:name, body without comments) of every __global__ function."""
    for path in SOURCES:
        with open(path) as f:
            text = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
        for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s*)?(\w+)\s*\(", text):
            start = text.index("{", m.end())
            depth, end = 1, start + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
            yield f"{os.path.basename(path)}:{m.group(1)}", text[start:end]


KERNELS = dict(_kernels())
WITH_TMEM = [k for k, body in KERNELS.items() if "tmem_alloc" in body]


def test_the_kernels_are_found():
    assert len(KERNELS) >= 15 and len(WITH_TMEM) >= 9, (sorted(KERNELS), WITH_TMEM)


@pytest.mark.parametrize("name", WITH_TMEM)
def test_tmem_is_taken_after_the_predecessors_have_ended(name):
    """A CTA that holds TMEM while it waits for its predecessors can starve one of them on its SM, which
    allocates only after it has let its dependents launch: neither would end."""
    body = KERNELS[name]
    assert body.count("grid_dependency_wait()") == 1
    assert body.index("grid_dependency_wait()") < body.index("tmem_alloc")
