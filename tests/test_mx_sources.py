"""What the compiler and a run cannot show: the microscaled kernels start before
the kernel ahead of them on the stream has ended, and any of their inputs may be
what that one writes.  The read-only data path (ld.global.nc, __ldg, or const
__restrict__ parameters, which the compiler may turn into it) is for data that
nothing writes while the kernel lasts, so none of their loads may take it, and
every kernel waits for the one ahead before its first load."""
import os
import re

import pytest

import mxfp4_routed_expert_k3mx_gb300 as k3mx

CSRC = os.path.join(os.path.dirname(k3mx.LIB_PATH), "csrc")


def code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"/\*.*?\*/", "", re.sub(r"//[^\n]*", "", text), flags=re.S)


@pytest.mark.parametrize("name", ["mxfmt.cu", "mxprod.cu"])
def test_inputs_are_not_read_through_the_read_only_path(name):
    text = code(name)
    assert "__global__" in text
    for word in ("__ldg", "ld.global.nc", "__restrict__"):
        assert word not in text, word


@pytest.mark.parametrize("name", ["mxfmt.cu", "mxprod.cu"])
def test_every_kernel_waits_for_the_one_ahead(name):
    kernels = code(name).split("__global__")[1:]
    assert len(kernels) == {"mxfmt.cu": 3, "mxprod.cu": 1}[name]
    for k in kernels:
        assert "pdl_wait()" in k and k.index("pdl_wait()") < k.index("pdl_launch_dependents()")
