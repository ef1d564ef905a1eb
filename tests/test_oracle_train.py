"""The oracle's training functions against other forms of the same: the plan
against the layer's, gradients against differences of the forward functions,
the optimizer against torch's, the 8-bit states against a search over codes."""

import numpy as np
import pytest
import torch

import oracle
from oracle import train as R


def _routing(rng, T, E, k):
    return np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)


@pytest.mark.parametrize("T,E,El,first,k", [(0, 4, 4, 0, 2), (1, 4, 4, 0, 1), (50, 8, 3, 2, 4), (300, 6, 6, 0, 2)])
def test_plan_is_the_compact_layout(T, E, El, first, k):
    rng = np.random.default_rng(T + E)
    ids = _routing(rng, T, E, k) if T else np.zeros((0, k), np.int32)
    if T > 2:
        ids[1, 0] = -1
    dst, start, counts = R.sort_plan(ids, E, El, first)
    plan = oracle.plan_layout(ids, E, El, first, "compact", 128, None)
    assert np.array_equal(dst.reshape(-1), np.asarray(plan["src2dst"]).reshape(-1))
    assert np.array_equal(counts, plan["counts"]) and np.array_equal(start, plan["start"])


def _difference(f, x, dout, h=1e-6):
    """Gradient of sum(f(x) * dout) by central differences."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        g[i] = (np.nansum(f(up) * dout) - np.nansum(f(down) * dout)) / (2 * h)
    return g


def test_row_gradients_by_differences():
    rng = np.random.default_rng(0)
    ids = _routing(rng, 5, 4, 2)
    ids[3] = -1
    dst, _, _ = R.sort_plan(ids, 4, 3, 0)
    rows = 3 * 128
    x, w = rng.standard_normal((5, 3)), rng.random((5, 2))
    dsorted = rng.standard_normal((rows, 3))
    zero = np.zeros((rows, 3))
    assert np.allclose(_difference(lambda a: R.sort_tokens(a, dst, zero), x, dsorted), R.unsort_tokens(dsorted, dst),
                       atol=1e-8)
    y, dout = rng.standard_normal((rows, 3)), rng.standard_normal((5, 3))
    dy, dw = R.unsort_tokens_backward(dout, y, dst, w, zero)
    assert np.allclose(_difference(lambda a: R.unsort_tokens(y, dst, a), w, dout), dw, atol=1e-8)
    used = dst[dst >= 0][:3]
    for d in used:
        def f(v, d=d):
            z = y.copy()
            z[d] = v
            return R.unsort_tokens(z, dst, w)
        assert np.allclose(_difference(f, y[d].copy(), dout), dy[d], atol=1e-8)


def test_product_gradients_by_differences():
    rng = np.random.default_rng(1)
    start, counts = np.array([0, 128, 128]), np.array([2, 0, 3])
    x, w = rng.standard_normal((131, 4)), rng.standard_normal((3, 5, 4))
    dy = rng.standard_normal((131, 5))
    dx = R.expert_gemm_dgrad(dy, w, start, counts)
    got = _difference(lambda a: R.expert_gemm(a, w, start, counts), x, dy)
    valid = np.r_[0:2, 128:131]
    assert np.allclose(got[valid], dx[valid], atol=1e-7)
    assert np.allclose(_difference(lambda a: R.expert_gemm(x, a, start, counts), w, dy),
                       R.expert_gemm_wgrad(dy, x, start, counts), atol=1e-7)
    gu, dh = rng.standard_normal((3, 8)) * 3, rng.standard_normal((3, 4))
    assert np.allclose(_difference(R.swiglu, gu, dh), R.swiglu_backward(dh, gu), atol=1e-7)


def test_adamw_is_torchs():
    rng = np.random.default_rng(2)
    p = torch.from_numpy(rng.standard_normal(50)).requires_grad_()
    opt = torch.optim.AdamW([p], lr=0.01, betas=(0.9, 0.95), eps=1e-6, weight_decay=0.1)
    mine, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for step in range(1, 6):
        g = rng.standard_normal(50)
        p.grad = torch.from_numpy(g.copy())
        opt.step()
        mine, m, v = R.adamw(mine, g, m, v, step, 0.01, 0.9, 0.95, 1e-6, 0.1)
        assert np.allclose(mine, p.detach().numpy(), rtol=1e-12, atol=1e-14)


def test_state_codes_are_the_nearest_roots():
    rng = np.random.default_rng(3)
    x = rng.standard_normal(600) ** 3
    s = R.state_scales(x)
    assert s.shape == (3,) and s[2] == np.abs(x[512:]).max()
    r = np.round(R.state_roots(x, 2, 127, s))
    every = R.state_values(np.arange(-127, 128), 2, 127, [1.0])
    for i in range(0, 600, 37):
        near = np.argmin(np.abs(np.sign(every) * np.sqrt(np.abs(every)) - np.sign(x[i]) * np.sqrt(abs(x[i]) / s[i // 256])))
        assert near - 127 == r[i]
    back = R.state_values(r, 2, 127, s)
    assert np.all(np.abs(back - x) <= np.abs(x) * 0.01 + np.sqrt(np.abs(x) * s.max()) * 0.009 + s.max() * 2e-5)
    assert not np.any(R.state_roots(np.zeros(10), 4, 255, R.state_scales(np.zeros(10))))
