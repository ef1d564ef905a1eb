"""Biases' gradients of small integers: every sum is exact in fp32 in whatever order, so a row that is lost or counted
twice shows (none is 0).  Rows around the steps of a CTA (128 or 256), of a cluster that shares an expert's rows (2, 4 and
8 CTAs), and of neither."""

import pytest
import torch

import moe_expert_layer_ep_gb300 as M

pytestmark = pytest.mark.gpu


def _rows(rows, N, seed):
    """-8 to 8 without 0, at most 8 * rows <= 2^24 a sum."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randint(1, 9, (rows, N), generator=g, device="cuda", dtype=torch.int8)
    v *= torch.randint(0, 2, (rows, N), generator=g, device="cuda", dtype=torch.int8) * 2 - 1
    return v.to(torch.bfloat16)


def _check(dy, start, counts):
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    at = [None if r is None else torch.tensor(r, dtype=torch.int32, device="cuda") for r in (start, counts)]
    db = M.moe_expert_bias_grad(dy, *at, status)
    for e, (s, n) in enumerate(zip(start or [0], counts or [dy.shape[0]])):
        assert torch.equal(db[e], dy[s:s + n].float().sum(0))
    again = M.moe_expert_bias_grad(dy, *at, status, db=db.clone(), accumulate=True)
    assert torch.equal(again, 2 * db) and int(status[0]) == 0


# N = 64 and 200: CTAs of 64 columns, whose rows two share from 1024 on, four from 2048, eight from 4096.
# N = 19456 and 9728: CTAs of 128 columns; two share from 512 rows on, four (of the latter) from 1024, eight from 2048.
@pytest.mark.parametrize("N,rows", [(64, n) for n in (1, 7, 31, 32, 33, 255, 256, 257, 1023, 1024, 1025, 1279, 1535, 2047, 2048, 2049,
                                                     3071, 3073, 4095, 4096, 4097, 6143, 6145, 9000, 65_537)]
                         + [(200, n) for n in (33, 1025, 2049, 4097)]
                         + [(19_456, n) for n in (1, 127, 129, 511, 512, 513, 639, 767, 769, 2000)]
                         + [(9_728, n) for n in (1024, 1025, 1151, 1535, 1537, 2047, 2048, 2049, 3071, 3073)]
                         + [(40_000, n) for n in (1, 17, 128, 255, 300)])
def test_dense(N, rows):
    _check(_rows(rows, N, rows + N), None, None)


@pytest.mark.parametrize("N,counts", [(64, [5000, 3, 0, 2600]), (72, [0, 4097, 1]), (64, [9001, 8999]), (136, [1, 0, 257, 255, 33] * 8),
                                      (4864, [1025, 513, 1, 600, 0, 511, 2049, 130]), (1536, [n % 700 for n in range(0, 12_800, 100)])])
def test_by_expert(N, counts):
    start, end = [], 3
    for n in counts:
        start.append(end)
        end += n + 5          # (rows of no expert between)
    _check(_rows(end, N, 90 + N), start, counts)


def test_past_32_bits_of_elements():
    dy = torch.empty((70_000, 32_768), dtype=torch.bfloat16, device="cuda")
    for a in range(0, 70_000, 10_000):
        dy[a:a + 10_000] = _rows(10_000, 32_768, a)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    db = M.moe_expert_bias_grad(dy, None, None, status)[0]
    want = torch.zeros(32_768, device="cuda")
    for a in range(0, 70_000, 10_000):
        want += dy[a:a + 10_000].float().sum(0)
    assert torch.equal(db, want)
