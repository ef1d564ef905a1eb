"""The training operators together, as the example runs them: a whole step's
gradients against torch's autograd on the same bf16 values, and a loss that
falls.

Tolerance of the gradients: the reference keeps every intermediate in fp64; the
layer rounds xs, gu, h, y, dy, dgu and the result to bf16, at most six roundings
of 2^-8 in a chain, each spread over sums of many terms: 6 * 2^-8 of the
gradient's norm.
"""

import os
import sys

import pytest
import torch

import synth

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import train_experts as X  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,K,I,E,topk", [(1, 64, 32, 4, 2), (77, 128, 96, 16, 3), (600, 256, 320, 8, 2)])
def test_gradients_of_a_step_are_autograds(T, K, I, E, topk):
    w13 = synth.bf16_expert_weights(E, 2 * I, K, 1, "cuda") * 4
    w2 = synth.bf16_expert_weights(E, K, I, 2, "cuda") * 4
    layer = X.ExpertLayer(w13, w2, T, topk)
    x = synth.activations(T, K, 3, "cuda")
    ids, weights = (t.cuda() for t in synth.routing(T, E, topk, 4))
    if T > 5:
        ids[5, 0] = -1
    dout = synth.activations(T, K, 5, "cuda")
    out = layer.forward(x, ids, weights).clone()
    got = [t.clone() for t in layer.backward(dout, weights)]

    leaves = [t.double().requires_grad_() for t in (w13, w2, x, weights)]
    a13, a2, ax, aw = leaves
    want = torch.zeros((T, K), dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(topk):
            e = int(ids[t, j])
            if e >= 0:
                g, u = (a13[e] @ ax[t]).chunk(2)
                want[t] = want[t] + aw[t, j] * (a2[e] @ (torch.nn.functional.silu(g) * u))
    ref = torch.autograd.grad((want * dout.double()).sum(), leaves)
    assert (out.double() - want).norm() <= 6 * 2.0 ** -8 * want.norm()
    for a, b in zip(got, ref):
        assert (a.double() - b).norm() <= 6 * 2.0 ** -8 * b.norm()


@pytest.mark.parametrize("bits", [8, 32])
def test_the_example_learns(bits):
    losses = X.train(steps=40, state_bits=bits)
    assert all(v == v for v in losses)
    assert sum(losses[-4:]) < 0.5 * sum(losses[:4])


def test_gradients_over_several_batches_add_up():
    T, K, I, E, topk = 200, 128, 96, 8, 2
    w13 = synth.bf16_expert_weights(E, 2 * I, K, 1, "cuda") * 4
    w2 = synth.bf16_expert_weights(E, K, I, 2, "cuda") * 4
    layer = X.ExpertLayer(w13, w2, T, topk, torch.float32)
    sums = None
    for part in range(3):
        x = synth.activations(T, K, 3 + part, "cuda")
        ids, weights = (t.cuda() for t in synth.routing(T, E, topk, 14 + part))
        layer.forward(x, ids, weights)
        dout = synth.activations(T, K, 25 + part, "cuda")
        kept = [layer.dw13.clone(), layer.dw2.clone()]
        one = [t.clone() for t in layer.backward(dout, weights)[:2]]
        sums = one if sums is None else [a + b for a, b in zip(sums, one)]
        if part > 0:
            layer.dw13.copy_(kept[0])
            layer.dw2.copy_(kept[1])
            layer.backward(dout, weights, accumulate=True)
        assert torch.equal(layer.dw13, sums[0]) and torch.equal(layer.dw2, sums[1])


def test_the_example_learns_from_several_batches_a_step():
    losses = X.train(steps=20, batches_per_step=2)
    assert all(v == v for v in losses)
    assert sum(losses[-2:]) < 0.5 * sum(losses[:2])
