"""Kernels that overlap their predecessor wait for it before they let the next one start, and do nothing in between:
only then has the kernel two places before one completed when it starts, and only a kernel's own wait makes visible
what it reads.  Read from the sources, without a GPU."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_expert_layer_ep_gb300", "csrc")


def _kernels():
    """(file:kernel, body without comments) of every kernel that takes part."""
    found = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__[^;{]*?(\w+)\s*\((?:[^(){};]|\([^(){};]*\))*\)\s*\{", text):
            depth, end = 1, m.end()
            while depth:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
            body = text[m.end():end]
            if "pdl_" in body:
                found.append((f"{os.path.basename(path)}:{m.group(1)}", body))
    return found


KERNELS = _kernels()


def test_the_kernels_are_found():
    assert len(KERNELS) >= 20


@pytest.mark.parametrize("name,body", KERNELS, ids=[k[0] for k in KERNELS])
def test_a_kernel_waits_and_then_triggers(name, body):
    assert len(re.findall(r"pdl_wait\(\)", body)) == 1 and len(re.findall(r"pdl_trigger\(\)", body)) == 1
    assert re.search(r"pdl_wait\(\);\s*pdl_trigger\(\);", body)
