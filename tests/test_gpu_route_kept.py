"""The router's gradient with dropped assignments that keep their ids, against the fp64 oracle and autograd.

Tolerances as in test_gpu_route_backward.py; a dropped assignment's part of the gradient is w times the sum of the kept
w dw, with the error that the kept ones' have."""

import os
import sys

import numpy as np
import pytest
import torch

import moe_expert_layer_ep_gb300 as M
import synth
from oracle import train as R

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_route_backward import BF, SIZES, Case, U, _f64  # noqa: E402

pytestmark = pytest.mark.gpu


class Kept(Case):
    def __init__(self, *args, lost=0.2, **kw):
        super().__init__(*args, **kw)
        g = torch.Generator().manual_seed(99 + self.T)
        self.kept = torch.rand((self.T, self.topk), generator=g) >= lost
        self.dtype = torch.uint8 if self.T % 2 else torch.bool

    def run(self, balance, zloss, **kw):
        return super().run(balance, zloss, kept=self.kept.to(self.dtype).cuda(), **kw)

    def reference(self, balance, zloss):
        z, ids, wt, dw = _f64(self.z), self.ids.numpy(), _f64(self.wt), _f64(self.dw)
        there, E = (ids >= 0).any(1), self.E
        kept = self.kept.numpy() & (ids >= 0)
        z, wt, dw = np.where(there[:, None], z, 0.0), np.where(ids >= 0, wt, 0.0), np.where(kept, dw, 0.0)
        dz = R.route_backward(z, ids, wt, dw, balance, zloss, kept)
        n = max(1, there.sum())
        f = np.bincount(ids[kept], minlength=E) / (n * self.topk)
        D = z.max(1, keepdims=True) - z
        p = np.exp(-D)
        lse = z.max(1, keepdims=True) + np.log(p.sum(1, keepdims=True))
        p = p / p.sum(1, keepdims=True)
        rp, rm, m = (D + E / 32 + 14) * U, (E / 32 + 30) * U, (f * p).sum(1, keepdims=True)
        cb, cz = balance * E / n, 2 * zloss / n
        near = cb * p * (rp * np.abs(f - m) + U * f + rm * m) + cz * p * ((rp + 2 * U) * np.abs(lse) + rm + U * np.abs(lse))
        sizes = cb * p * np.abs(f - m) + cz * p * np.abs(lse)
        total = np.abs(wt * dw).sum(1)
        for t, j in zip(*np.nonzero(ids >= 0)):
            pull = wt[t, j] * (abs(dw[t, j]) + total[t])
            near[t, ids[t, j]] += 12 * U * pull
            sizes[t, ids[t, j]] += pull
        near = np.where(there[:, None], near + 2 * U * sizes, 0.0)
        losses = np.array(R.route_losses(z, ids, kept))
        off = np.array([losses[0] * (E / 32 + 60) * U, (2 * np.abs(lse[there]) * (rm + U * np.abs(lse[there]))).sum() / n
                        + 4 * U * losses[1]])
        return dz, near, losses, off + 1e-30


@pytest.mark.parametrize("T,K,E,topk", SIZES)
def test_gradient_matches_the_oracle(T, K, E, topk):
    c = Kept(T, K, E, topk, 2000 + T + E, drop=0.1 if T > 5 else 0.0)   # (ids of -1 among them)
    if T > 50:
        c.kept[31] = False
    c.check(0.7, 0.3, residual=T % 2 == 0)
    c.check(0.0, 0.0, residual=T % 2 == 1)


def test_a_dropped_assignments_gradient_is_not_read():
    c = Kept(150, 256, 72, 4, 11, pad=23)
    want = c.check(0.5, 0.2)
    c.dw[~c.kept] = float("nan")
    for a, b in zip(c.run(0.5, 0.2), want):
        assert torch.equal(a, b)


def test_all_kept_and_none():
    c = Kept(130, 256, 40, 4, 12, lost=0.0)
    assert c.kept.all()
    plain = Case(130, 256, 40, 4, 12)
    for a, b in zip(c.run(0.5, 0.2), plain.run(0.5, 0.2)):
        assert torch.equal(a, b)
    c.kept[:] = False        # no selection, no load: the logits' size alone
    dx, dw, losses, dz = c.check(0.5, 0.2)
    assert losses[0] == 0 and losses[1] > 0 and dz.any()
    assert not c.run(0.5, 0.0)[3].any()


def test_a_layer_that_drops_assignments():
    """moe_route's ids and weights, some assignments dropped before the plan, the gradients of the sorted layer's calls:
    autograd's in fp64 through a softmax over all selections and a mask.  Bounds as where nothing is dropped: dx within
    one bf16 rounding and what fp32 logits lose, 2^-8 + 1e-4 of its norm, dW within 1e-4."""
    T, K, E, k = 500, 512, 64, 6
    x = synth.activations(T, K, 21, "cuda")
    w = torch.randn((E, K), generator=torch.Generator().manual_seed(22)).cuda() * 0.1
    planes = M.moe_router_prepare(w)
    ids, wt, z = M.moe_route(x, planes, k)
    lost = (torch.rand((T, k), generator=torch.Generator().manual_seed(24)) < 0.1).cuda()
    kept = M.moe_sort_plan(ids.masked_fill(lost, -1), E)[0] >= 0
    assert torch.equal(kept, ~lost)
    dwt = torch.randn((T, k), generator=torch.Generator().manual_seed(23)).cuda() + 0.3
    dx, dw, losses = M.moe_route_backward(x, planes, z, ids, wt, dwt, balance=3.0, zloss=0.5, kept=kept)
    ax, aw = x.double().requires_grad_(), w.double().requires_grad_()
    logits = ax @ aw.T
    sel = torch.softmax(logits.gather(1, ids.long()), 1).masked_fill(lost, 0.0)
    f = torch.bincount(ids[~lost].long(), minlength=E).double() / (T * k)
    b = E * (f * torch.softmax(logits, 1).mean(0)).sum()
    s = (torch.logsumexp(logits, 1) ** 2).mean()
    rx, rw = torch.autograd.grad((sel * dwt.double()).sum() + 3.0 * b + 0.5 * s, (ax, aw))
    assert (dx.double() - rx).norm() <= (BF + 1e-4) * rx.norm()
    assert (dw.double() - rw).norm() <= 1e-4 * rw.norm()
    assert torch.allclose(losses.double(), torch.stack((b, s)), rtol=1e-5)


def test_captured_and_on_another_stream():
    c = Kept(700, 256, 96, 4, 16)
    args, kept = c.args(), c.kept.cuda()
    ws = torch.empty(M.moe_route_backward_workspace_size(c.T, c.K, c.E), dtype=torch.uint8, device="cuda")

    def run(stream=None):
        return M.moe_route_backward(*args, balance=0.3, zloss=0.1, ws=ws, stream=stream, kept=kept)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    kept.logical_not_()      # a replay reads what is there then
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in out]
    side = torch.cuda.Stream()
    want = run(side)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_refusals():
    c = Kept(20, 256, 16, 2, 25)
    a, kept = c.args(), c.kept.cuda()
    for bad in (kept.int(), kept[:, :1].contiguous(), kept.cpu(), kept.float(), kept[::2]):
        with pytest.raises(ValueError):
            M.moe_route_backward(*a, kept=bad)
