"""The AdamW step's own root and reciprocal against CUDA's rounded ones, over every
number of every binade that they are used on (tests/native/adamw_math.cu)."""

import ctypes
import os
import subprocess

import pytest
import torch

from moe_expert_layer_ep_gb300 import build

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def compare(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("native") / "adamw_math.so")
    subprocess.run([build.nvcc(), *build.ARCH, "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-I",
                    os.path.join(build.ROOT, "include"), os.path.join(HERE, "native", "adamw_math.cu"), "-o", lib],
                   check=True)
    fn = ctypes.CDLL(lib).adamw_compare
    fn.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_void_p]

    def call(what, e):
        out = torch.zeros(2, dtype=torch.int64, device="cuda")
        torch.cuda.synchronize()
        assert fn(what, e, out.data_ptr()) == 0
        return out.tolist()

    return call


def test_roots_are_the_rounded_ones(compare):
    """From 2^-100 up; below, where the residual of the Newton step may be subnormal, one ulp off at most."""
    assert all(compare(0, e) == [0, 0] for e in range(-100, 128))
    assert all(compare(0, e)[1] <= 1 for e in range(-126, -100))


def test_reciprocals_are_within_two_ulps(compare):
    """Of numbers whose reciprocal is normal."""
    assert all(compare(1, e)[1] <= 2 for e in range(-126, 126))
