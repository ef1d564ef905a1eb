"""The benchmark's write-only bandwidth is the memory's, not a kernel's."""

import pytest
import torch

import bench

pytestmark = pytest.mark.gpu


def _gbs(f, nbytes):
    for _ in range(3):
        f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(10):
        f()
    b.record()
    torch.cuda.synchronize()
    return 10 * nbytes / (a.elapsed_time(b) / 1e3) / 1e9


def test_write_peak_is_not_below_what_clearing_memory_reaches():
    """A stream of writes cannot be slower than one of writes that is there; 15 % for noise between two timings."""
    buf = torch.empty(512 << 20, dtype=torch.uint8, device="cuda")
    clear = max(_gbs(buf.view(torch.float64).zero_, buf.numel()) for _ in range(3))
    assert max(bench.measure_write_peak("cuda") for _ in range(3)) >= 0.85 * clear
