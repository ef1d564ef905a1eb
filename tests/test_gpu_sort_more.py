"""Tokens sorted by expert and back: the rows' gradient without the weights'."""

import pytest
import torch

import moe_expert_layer_ep_gb300 as M

pytestmark = pytest.mark.gpu


def _routing(T, E, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.topk(torch.rand((T, E), generator=g, device="cuda"), k).indices.to(torch.int32)
    ids[torch.rand((T, k), generator=g, device="cuda") < 0.1] = -1
    return ids, torch.rand((T, k), generator=g, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K,k", [(1, 8, 1), (77, 1001, 8), (300, 130, 11), (513, 2048, 4), (40, 1002, 3)])
def test_rows_gradient_alone(T, K, k, dtype):
    """The same bits as beside the weights' gradient, and nothing but the tokens' rows is written."""
    E = 16
    ids, w = _routing(T, E, k, T)
    s2d, _, _ = M.moe_sort_plan(ids, E)
    rows = M.moe_compact_all_tokens(T * k, E)
    g = torch.Generator(device="cuda").manual_seed(K)
    dout, y = (torch.randn((n, K), generator=g, device="cuda").to(dtype) for n in (T, rows))
    want, _ = M.moe_unsort_tokens_backward(dout, y, s2d, w, dy=torch.full_like(y, 7.0))
    got = torch.full_like(y, 7.0)
    dy, dw = M.moe_unsort_tokens_backward(dout, None, s2d, w, dy=got)
    assert dy is got and dw is None and torch.equal(got, want)
    at = s2d[s2d >= 0].long()
    dy, dw = M.moe_unsort_tokens_backward(dout, None, s2d, w, rows=rows)
    assert dw is None and dy.shape == y.shape and torch.equal(dy[at], want[at])
    # the formula itself
    ref = torch.zeros((rows, K), dtype=torch.float64, device="cuda")
    for j in range(k):
        kept = s2d[:, j] >= 0
        ref[s2d[kept, j].long()] = w[kept, j, None].double() * dout[kept].double()
    near = 2.0 ** -24 + (2.0 ** -8 * 1.001 if dtype == torch.bfloat16 else 0.0)
    assert torch.all((got[at].double() - ref[at]).abs() <= near * ref[at].abs())


def test_rows_gradient_alone_refusals_and_no_rows():
    dst = torch.arange(4, dtype=torch.int32, device="cuda").view(4, 1)
    x, w = torch.ones((4, 16), device="cuda"), torch.ones((4, 1), device="cuda")
    for bad in (dict(), dict(dw=w, rows=4), dict(dy=x[:, :8]), dict(dy=x.bfloat16()), dict(dy=x, rows=5), dict(dy=x[0])):
        with pytest.raises(ValueError):
            M.moe_unsort_tokens_backward(x, None, dst, w, **bad)
    with pytest.raises(ValueError):
        M.moe_unsort_tokens_backward(x, x, dst, w, rows=5)
    dy, dw = M.moe_unsort_tokens_backward(x, None, torch.full_like(dst, -1), w, rows=0)
    assert dy.shape == (0, 16) and dw is None
