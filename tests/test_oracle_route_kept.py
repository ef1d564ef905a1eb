"""Pins of the router's gradient where assignments were dropped: torch's derivative in fp64."""

import numpy as np
import pytest
import torch

from oracle import train as R


def _autograd(z, ids, kept, dw, cb, cz, over):
    """Of cb * balance + cz * size + sum over the kept of dw * w, w the softmax over the assignments `over`."""
    T, E = z.shape
    k = ids.shape[1]
    zz = torch.tensor(z, requires_grad=True)
    at, keep, over = torch.tensor(ids).clamp(min=0), torch.tensor(kept), torch.tensor(over)
    there = over.any(1)
    n = int(there.sum())
    w = torch.softmax(zz.gather(1, at).masked_fill(~over, -1e300), 1)
    f = torch.bincount(at[keep], minlength=E).double() / (n * k)
    p = torch.softmax(zz, 1)[there]
    balance, size = E * (f * p.mean(0)).sum(), (torch.logsumexp(zz, 1)[there] ** 2).mean()
    total = cb * balance + cz * size + (w * torch.tensor(dw))[keep].sum()
    return w.detach().numpy(), torch.autograd.grad(total, zz)[0].numpy(), (float(balance.detach()), float(size.detach()))


@pytest.mark.parametrize("mean", [0.0, 0.3])
def test_dropped_assignments(mean):
    rng = np.random.default_rng(5)
    T, E, k = 60, 16, 4
    z = rng.normal(size=(T, E))
    ids = np.argsort(-z, 1)[:, :k].copy()
    dw = rng.normal(size=(T, k)) * 0.1 + mean
    kept = rng.random((T, k)) > 0.2
    kept[7] = False          # all dropped: a token all the same
    # weights over all selected, ids as they were
    w, want, losses = _autograd(z, ids, kept, dw, 0.7, 0.3, np.ones((T, k), bool))
    got = R.route_backward(z, ids, w, np.where(kept, dw, np.nan), 0.7, 0.3, kept)
    assert np.abs(got - want).max() < 1e-12
    assert np.allclose(R.route_losses(z, ids, kept), losses, rtol=1e-13)
    # a token's gradient through a softmax sums to 0; with the ids gone, that of these weights would not
    alone = R.route_backward(z, ids, w, dw, 0.0, 0.0, kept)
    gone = R.route_backward(z, np.where(kept, ids, -1), w, dw, 0.0, 0.0)
    assert np.abs(alone.sum(1)).max() < 1e-12 and np.abs(gone.sum(1)).max() > 1e-3
    # weights over those that are left, the others' ids -1
    left = np.where(kept, ids, -1)
    w, want, losses = _autograd(z, left, kept, dw, 0.7, 0.3, kept)
    there = kept.any(1)
    got = R.route_backward(z, left, np.where(kept, w, 0.0), dw, 0.7, 0.3)
    assert np.abs(got - want)[there].max() < 1e-12 and not got[~there].any()
    assert np.allclose(R.route_losses(z, left), losses, rtol=1e-13)
