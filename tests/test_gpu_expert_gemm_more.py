"""The experts' products where their numbers are at an end: last rows that are
cleared between the two CTAs of a pair, tiles of every height, reductions that
take seconds, no rows at all.
"""

import pytest
import torch

import moe_expert_layer_ep_gb300 as M

pytestmark = pytest.mark.gpu


def _randn(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + sum(shape))
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def _at(start, counts):
    at = [torch.as_tensor(v, dtype=torch.int32, device="cuda") for v in (start, counts)]
    return (*at, torch.zeros(4, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("N,C", [(256, 256), (520, 88), (136, 640)])
def test_cleared_last_rows_are_those_of_zeros(N, C):
    """Experts of 1 to 200 rows among rows of NaN, against the same rows followed by zeros up to whole blocks of 64,
    which no clearing touches: zeros add nothing, so the same bits, call after call."""
    E, step = 200, 256
    counts = torch.arange(1, E + 1)
    dy, x = _randn(E * step, N), _randn(E * step, C)
    row = torch.arange(E * step, device="cuda")
    past = (row % step) >= (row // step + 1)
    zeros = [t.masked_fill(past[:, None], 0.0) for t in (dy, x)]
    nans = [t.masked_fill(past[:, None], float("nan")) for t in (dy, x)]
    start = torch.arange(E) * step
    want = M.moe_expert_gemm_wgrad(*zeros, *_at(start, (counts + 63) // 64 * 64))
    at = _at(start, counts)
    for _ in range(30):
        assert torch.equal(M.moe_expert_gemm_wgrad(*nans, *at), want)
    assert torch.isfinite(want).all() and int(at[2][0]) == 0
