"""The example's step over several batches has the gradient of their mean, the router's losses included: B copies of one
batch give that of one.  1 / B is a power of two here, so every term is scaled exactly, and what differs is the order of
at most B * parts + 1 additions of dW (parts <= 2 for 512 tokens): 10 * 2^-24 of sums that are about dW's size, taken as
1e-5 of its norm."""

import os
import sys

import pytest
import torch

import moe_expert_layer_ep_gb300 as M
import synth

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import train_experts as X  # noqa: E402

pytestmark = pytest.mark.gpu


def test_copies_of_a_batch_have_its_gradient(monkeypatch):
    activations = synth.activations
    monkeypatch.setattr(synth, "activations", lambda T, K, seed, device: activations(T, K, 5, device))
    create = M.moe_adamw_create
    seen = []

    def watched(params, grads, *args, **kwargs):
        seen.append(grads)
        return create(params, grads, *args, **kwargs)

    monkeypatch.setattr(M, "moe_adamw_create", watched)
    got = []
    for batches in (1, 2, 4):
        X.train(steps=1, train_router=True, batches_per_step=batches)
        got.append([g.float().clone() for g in seen[-1]])
    for w13, w2, router in got[1:]:
        assert (router - got[0][2]).norm() <= 1e-5 * got[0][2].norm()
        for a, b in zip((w13, w2), got[0]):       # (one batch's are stored in bf16)
            assert (a - b).norm() <= 2.0 ** -8 * b.norm()
