"""The timing calls' kernel names: the sources' kernels, every one of them (CPU)."""
import glob
import os
import re

import pytest

from mesa_layer_gb300 import binding, build


@pytest.fixture(scope="module")
def names():
    build.build()
    lib = binding.load()
    lib.mesa_kernel_name.restype = binding.ctypes.c_char_p
    found, i = [], 0
    while True:
        name = lib.mesa_kernel_name(i)
        if name is None:
            return found
        found.append(name.decode())
        i += 1


def test_kernels_of_the_scan_the_convolution_and_the_rotation(names):
    listed = {n for kind in names for n in kind.split("|")}
    for path in glob.glob(os.path.join(build.CSRC, "*.cu")):
        if os.path.basename(path).startswith(("ssm", "causal_conv", "qk_rotary")):
            text = open(path).read()
            kernels = set(re.findall(r"__global__[^;{]*?\b(mesa_\w+_kernel)\(", text))
            assert kernels and kernels <= listed, (path, kernels - listed)


def test_no_kernel_is_named_that_is_not_there(names):
    text = "".join(open(p).read() for p in glob.glob(os.path.join(build.CSRC, "*.cu*")))
    there = set(re.findall(r"__global__[^;{]*?\b(\w+)\s*\(", text)) | set(re.findall(r"\b(mesa_\w+_kernel)\s*\(", text))
    assert {n.split("<")[0] for kind in names for n in re.split(r"[|+]", kind)} <= there
