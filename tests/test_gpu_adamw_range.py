"""AdamW at the ends of fp32's range: gradients whose square is beyond it, second
moments that are infinite or not numbers.

Where v is infinite the step is m / inf = 0 and the parameter only decays: one
product with a rounded constant, 2 U |p| off at most (U = 2^-24).  Elements that
have nothing to do with such a value keep the bits that they have without it.
"""

import numpy as np
import pytest
import torch

import moe_expert_layer_ep_gb300 as M
from test_gpu_adamw import HYPER, U, Tensor, _create, _f64

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
KINDS = [("fp32", "fp32", False), ("bf16", "bf16", True), ("bf16", "fp32", False)]
kinds = pytest.mark.parametrize("param,grad,master", KINDS)


def _decayed(before, after, at, steps=1, hyper=HYPER):
    """The values that are stepped, at the places `at`, are those of `before` after that many decays."""
    p, w = (_f64(t.p if t.w is None else t.w)[at] for t in (before, after))
    want = p * (1 - hyper["lr"] * hyper["weight_decay"]) ** steps
    store = 2.0 ** -8 * steps if after.w is None and after.p.dtype == torch.bfloat16 else 0.0
    assert np.all(np.abs(w - want) <= (2 * U * steps + store) * np.abs(p))


@kinds
@pytest.mark.parametrize("bits", [32, 8])
def test_a_gradient_whose_square_is_beyond_fp32(param, grad, master, bits):
    t = Tensor(1100, param, grad, bits, master, 3)
    plain = t.clone()
    huge = [10, 300, 301, 1099]
    t.g[huge] = torch.tensor([1e20, -3e38, 1.9e19, -1e25], device="cuda").to(t.g.dtype)
    before = t.clone()
    M.moe_adamw_step(_create([t]), **HYPER)
    M.moe_adamw_step(_create([plain]), **HYPER)
    torch.cuda.synchronize()
    assert torch.isfinite(t.p).all()
    _decayed(before, t, huge)
    rest = torch.ones(1100, dtype=torch.bool, device="cuda")
    rest[huge] = False
    assert torch.equal(t.p[rest], plain.p[rest])
    if master:
        assert torch.equal(t.w[rest], plain.w[rest])
    if bits == 32:
        assert torch.isinf(t.v[huge]).all() and torch.isfinite(t.m).all()
        assert torch.equal(t.v[rest], plain.v[rest]) and torch.equal(t.m[rest], plain.m[rest])
    else:
        assert torch.isinf(t.vs.cpu()).tolist() == [True, True, False, False, True] and torch.isfinite(t.ms).all()
        assert torch.equal(t.v[512:1024], plain.v[512:1024]) and torch.equal(t.m[512:1024], plain.m[512:1024])
        assert torch.all(t.v[huge] >= 1)
    # later steps with ordinary gradients: an infinite second moment stays so
    t.g.copy_(plain.g)
    stuck = rest.logical_not() if bits == 32 else torch.repeat_interleave(torch.isinf(t.vs), 256)[:1100] & (t.v > 0)
    at = stuck.nonzero().flatten().cpu().numpy()
    mid = t.clone()
    for step in (8, 9, 10):
        M.moe_adamw_step(_create([t]), **dict(HYPER, step=step))
        torch.cuda.synchronize()
        for x in t.all():
            assert not torch.isnan(x.float()).any()
        assert torch.isfinite(t.p).all()
    _decayed(mid, t, at, steps=3)


def test_a_huge_first_moment_and_a_long_step():
    """lr / (1 - beta1^t) * m is beyond fp32, m / inf is 0."""
    t = Tensor(300, "fp32", "fp32", 32, False, 4, zero=True)
    t.g[7] = 3e38
    before = t.clone()
    h = dict(HYPER, step=1, lr=5.0)
    M.moe_adamw_step(_create([t]), **h)
    torch.cuda.synchronize()
    assert torch.isfinite(t.p).all()
    _decayed(before, t, [7], hyper=h)


@pytest.mark.parametrize("bits", [32, 8])
def test_an_infinite_second_moment_is_no_step(bits):
    t = Tensor(600, "fp32", "fp32", bits, False, 5)
    plain = t.clone()
    if bits == 32:
        t.v[[5, 599]] = INF
        at = [5, 599]
    else:
        # a code 0 is v = 0 whatever its block's scale: an element of its own step
        t.vs[1] = INF
        t.v[256:300] = 0
        plain.vs[1], plain.v[256:300] = 1.0, 0
        at = [i for i in range(300, 512) if int(t.v[i]) > 0]
        assert len(at) > 100
    before = t.clone()
    M.moe_adamw_step(_create([t]), **HYPER)
    M.moe_adamw_step(_create([plain]), **HYPER)
    torch.cuda.synchronize()
    assert torch.isfinite(t.p).all()
    _decayed(before, t, at)
    rest = torch.ones(600, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(t.p[rest], plain.p[rest])


@pytest.mark.parametrize("bits", [32, 8])
def test_a_second_moment_that_is_no_number_is_seen(bits):
    t = Tensor(600, "fp32", "fp32", bits, False, 6)
    if bits == 32:
        t.v[[5, 599]] = NAN
        bad = [5, 599]
    else:
        t.vs[1] = NAN
        t.v[256:300] = 0
        bad = list(range(256, 512))
    M.moe_adamw_step(_create([t]), **HYPER)
    torch.cuda.synchronize()
    assert torch.isnan(t.p.cpu()).nonzero().flatten().tolist() == bad
    if bits == 32:
        assert torch.isnan(t.v.cpu()).nonzero().flatten().tolist() == bad
    else:
        assert torch.isnan(t.vs.cpu()).tolist() == [False, True, False]


@pytest.mark.parametrize("bad", [INF, -INF, NAN])
@pytest.mark.parametrize("bits", [32, 8])
def test_a_gradient_that_is_not_finite(bits, bad):
    """Its element at once, and in 8 bits its block's states from then on; no others."""
    t = Tensor(600, "fp32", "fp32", bits, False, 7)
    good = t.g.clone()
    t.g[300] = bad
    M.moe_adamw_step(_create([t]), **HYPER)
    torch.cuda.synchronize()
    assert (~torch.isfinite(t.p.cpu())).nonzero().flatten().tolist() == [300]
    if bits == 8:
        assert (~torch.isfinite(t.ms.cpu())).tolist() == [False, True, False]
    t.g.copy_(good)
    M.moe_adamw_step(_create([t]), **dict(HYPER, step=8))
    torch.cuda.synchronize()
    want = [300] if bits == 32 else list(range(256, 512))
    assert (~torch.isfinite(t.p.cpu())).nonzero().flatten().tolist() == want
