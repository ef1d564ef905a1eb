"""dx of the router's gradient where the rows of W have something in common, which cancels in a dz that sums to 0.

W_e = W'_e + a_e m, with m, per column, the middle of four evenly spread experts' values (of their first bf16 plane: half
the second and third in order, rounded to bf16) and a_e = 1 where that makes the sum of a row's sizes less than 0.7 of what it is; then dx = dz W' + (sum over a_e = 1 of dz_e) m.  Tolerance, U = 2^-23,
an fp32 operation 2^-24: W' and dz are taken with 11 bits (2^-10 of sum |dz W'| for both, 1.01 for their product and,
where a_e = 0, the plane of W that is left out, 2^-17 of W), the sum over the experts with (E / 16 + 16) U; W' is rounded
to fp32 from W and m (U (|W| + |m|)); the sum of dz is off by (E / 32 + 8) U of its sizes, its product with m and their addition by U; what dz itself is off, as in test_gpu_route_backward.py; 2^-37 E
of the largest term for values that are subnormal in fp16; and one rounding to bf16."""

import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_route_backward import BF, Case, U, _f64  # noqa: E402

pytestmark = pytest.mark.gpu


def _check(c, balance, zloss, residual=False):
    dz, near, _, _ = c.reference(balance, zloss)
    dx = _f64(c.run(balance, zloss, residual=c.res.cuda() if residual else None)[0])
    w, E = _f64(c.w), c.E
    four = c.w.to(torch.bfloat16).float()[[n * E // 4 for n in range(4)]].sort(dim=0).values
    m = _f64((0.5 * four[1] + 0.5 * four[2]).to(torch.bfloat16))
    am = np.abs(m)
    was, left = np.abs(w).sum(1), np.abs(w - m).sum(1)
    assert not np.any(np.abs(left - 0.7 * was) < 1e-4 * was)   # no row at the rule's edge
    centred = left < 0.7 * was
    rest = np.where(centred[:, None], w - m, w)
    ref, adz = dz @ w, np.abs(dz)
    part, total = np.where(centred, dz, 0.0).sum(1, keepdims=True), np.where(centred, adz, 0.0).sum(1, keepdims=True)
    size = adz @ np.abs(rest)
    A = (1.01 * 2.0 ** -10 + (E / 16 + 16) * U) * size + 2.0 ** -37 * E * (adz * np.abs(rest).max(1)).max(1, keepdims=True)
    A = A + near @ (np.abs(rest) + np.where(centred[:, None], am, 0.0))
    A = A + adz @ np.where(centred[:, None], U * (np.abs(w) + am), 0.0)
    A = A + ((E / 32 + 10) * U * total + 2 * U * np.abs(part)) * am + 2 * U * np.abs(ref)
    if residual:
        r = _f64(c.res)
        ref = ref + r
        A = A + U * (np.abs(ref) + np.abs(r))
    assert np.all(np.abs(dx - ref) <= A + BF * (np.abs(ref) + A) + 1e-37)
    return centred


def _with_row(T, K, E, topk, seed, size, which=slice(None)):
    c = Case(T, K, E, topk, seed)
    c.w[which] += 0.05 * size * torch.randn(K, generator=torch.Generator().manual_seed(seed))
    return c


@pytest.mark.parametrize("T,K,E,topk", [(1, 128, 4, 2), (64, 256, 128, 8), (300, 384, 37, 6), (1000, 2048, 128, 8), (129, 7168, 256, 8),
                                        (5, 256, 900, 64), (2049, 640, 65, 2)])
@pytest.mark.parametrize("size", [4.0, 32.0])
def test_a_common_row(T, K, E, topk, size):
    c = _with_row(T, K, E, topk, 3000 + T + E, size)
    assert _check(c, 0.7, 0.3, residual=T % 2 == 0).all()
    assert _check(c, 0.0, 0.0, residual=T % 2 == 1).all()
    _check(c, 1.0, 0.0)


def test_common_to_some_experts():
    c = _with_row(200, 512, 96, 6, 41, 20.0, slice(0, 80))
    centred = _check(c, 0.5, 0.5)
    assert centred[:80].all() and not centred[80:].any()


def test_beside_an_expert_of_large_weights():
    """Beside one, or one that has a few large values, the others' common row is found all the same; beside two of the
    four, the row is left alone where it would not help."""
    c = _with_row(200, 512, 64, 6, 42, 8.0)
    c.w[16] *= 1e5                 # one of the four that it is formed of
    c.z[:, 16] = float("-inf")      # and it is never chosen: its dz is 0
    v, ids = torch.topk(c.z, 6, dim=1)
    c.ids, c.wt = ids.to(torch.int32), torch.softmax(v, 1)
    others = torch.arange(64) != 16
    assert _check(c, 0.5, 0.5)[others].all()
    c.w[16] /= 1e5
    c.w[16, ::50] += 300.0
    assert _check(c, 0.5, 0.5)[others].all()
    c.w[[16, 32]] *= 1e5
    assert not _check(c, 0.5, 0.5)[torch.arange(64) % 16 != 0].any()


def test_one_expert_and_two():
    one = _with_row(70, 256, 1, 1, 43, 3.0)
    assert _check(one, 0.5, 0.5).all()
    _check(_with_row(70, 256, 2, 1, 44, 3.0), 0.5, 0.5)


def test_the_error_does_not_grow_with_what_is_common():
    """Of the norm, without a residual.  A rounding's error is spread evenly over half a step either way, so its root mean
    square is 1 / sqrt 3 of the largest: 2^-8 / sqrt 3 of a value for the store in bf16, and sqrt(2 / 3) 2^-11 of the
    terms' root sum of squares for the two factors, less than 2^-11.  (A common row 8 or 32 times the rest, rounded with
    it: 2.9e-3 and 9.7e-3.)"""
    for size in (0.0, 1.0, 8.0, 32.0):
        c = _with_row(2000, 512, 128, 8, 45, size)
        dz = c.reference(0.0, 0.0)[0]
        want = dz @ _f64(c.w)
        dx = _f64(c.run(0.0, 0.0)[0])
        assert np.linalg.norm(dx - want) <= (2.0 ** -8 / 3 ** 0.5 + 2.0 ** -11) * np.linalg.norm(want)


def test_a_tokens_bits_do_not_depend_on_the_others():
    c = _with_row(600, 384, 48, 4, 46, 16.0)
    few = Case(600, 384, 48, 4, 46)
    few.w = c.w
    keep = slice(300, 301)
    for name in ("x", "z", "ids", "wt", "dw", "res"):
        setattr(few, name, getattr(c, name)[keep].contiguous())
    few.T = 1
    a, b = c.run(0.0, 0.0)[0], few.run(0.0, 0.0)[0]
    assert torch.equal(a[keep].view(torch.int16), b.view(torch.int16))
