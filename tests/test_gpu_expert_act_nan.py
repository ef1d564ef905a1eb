"""A NaN before an activation is one in its value and in its gradient, and nowhere else."""

import pytest
import torch

import moe_expert_layer_ep_gb300 as M

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", [a for a in M.MOE_ACTS if a != "none"])
@pytest.mark.parametrize("dense", [True, False])   # few tiles; tiles of 256 features
def test_gradients_at_nan(act, dense):
    rows, N, C = 70, 64, 136
    g = torch.Generator(device="cuda").manual_seed(71)
    dy, w, gu = (torch.randn(s, generator=g, device="cuda").to(torch.bfloat16) for s in ((rows, N), (1, N, C), (rows, 2 * C)))
    at = [torch.tensor([v], dtype=torch.int32, device="cuda") for v in (0, rows)]
    at = ([None, None] if dense else at) + [torch.zeros(4, dtype=torch.int32, device="cuda")]
    places = torch.zeros((rows, C), dtype=torch.bool, device="cuda")
    places[0, 0] = places[33, 7] = places[69, 135] = places[64, 128] = True
    gu[:, :C][places] = float("nan")
    z = gu[:, :C].contiguous()
    assert torch.equal(M.moe_expert_gemm_dgrad_act(dy, w, *at, z=z, act=act).isnan(), places)
    assert torch.equal(M.moe_expert_gemm_dgrad_act(dy, w, *at, z=z, act=act, residual=z.nan_to_num()).isnan(), places)
    d = M.moe_expert_gemm_dgrad_glu(dy, w, gu, *at, act=act)
    assert torch.equal(d[:, :C].isnan(), places) and torch.equal(d[:, C:].isnan(), places)
    # and values
    x = torch.randn((rows, C), generator=g, device="cuda").to(torch.bfloat16)
    x[5, 3] = float("nan")
    y, _ = M.moe_expert_gemm_act(x, w, *at, act=act)
    h, _ = M.moe_expert_gemm_glu(x, w, *at, act=act)
    for t in (y, h):
        assert t[5].isnan().all() and not t[:5].isnan().any() and not t[6:].isnan().any()
