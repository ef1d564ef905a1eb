"""The training operators where element offsets pass 32 bits: sorted rows of more
than 2^31 elements and an optimizer tensor of more than 2^31, each against the
same operator on the few rows (elements) concerned, which other tests compare
with the oracle.  The results have to be the same bits.
"""

import pytest
import torch

import moe_expert_layer_ep_gb300 as M

pytestmark = pytest.mark.gpu


def _randn(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def test_sort_and_back_past_32_bits():
    T, K, E, k = 40000, 7168, 64, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.topk(torch.rand((T, E), generator=g, device="cuda"), k).indices.to(torch.int32)
    w = torch.rand((T, k), generator=g, device="cuda")
    x = _randn((T, K), 2)
    src2dst, start, counts = M.moe_sort_plan(ids, E)
    rows = M.moe_compact_all_tokens(T * k, E)
    assert rows * K > 2 ** 31 and int(src2dst.max()) * K > 2 ** 31
    y = M.moe_sort_tokens(x, src2dst, rows)
    for j in range(k):
        for t0 in range(0, T, 10000):   # a few GB at a time
            assert torch.equal(y[src2dst[t0:t0 + 10000, j].long()], x[t0:t0 + 10000])
    # the tokens whose rows lie furthest back, alone: their rows gathered into a small buffer
    some = torch.topk(src2dst.max(1).values, 50).indices
    near = y[src2dst[some].reshape(-1).long()].contiguous()
    dst = torch.arange(50 * k, dtype=torch.int32, device="cuda").view(50, k)
    assert torch.equal(M.moe_unsort_tokens(y, src2dst, w)[some], M.moe_unsort_tokens(near, dst, w[some].contiguous()))
    dout = _randn((T, K), 3)
    dy, dw = M.moe_unsort_tokens_backward(dout, y, src2dst, w)
    dy50, dw50 = M.moe_unsort_tokens_backward(dout[some].contiguous(), near, dst, w[some].contiguous())
    assert torch.equal(dy[src2dst[some].reshape(-1).long()], dy50) and torch.equal(dw[some], dw50)


def test_products_past_32_bits():
    rows, N, C, n = 2 ** 19 + 77, 4608, 4616, 100
    assert rows * N > 2 ** 31
    far = torch.tensor([0, rows - n], dtype=torch.int32, device="cuda")
    near = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    counts = torch.tensor([n, n], dtype=torch.int32, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    w13, w2 = _randn((2, 2 * N, 64), 4) * 0.1, _randn((2, 64, N), 5) * 0.1
    wide, wx = _randn((2, 72, C), 6), torch.empty((rows, C), dtype=torch.bfloat16, device="cuda")
    pick = torch.cat([torch.arange(n), torch.arange(rows - n, rows)]).cuda()
    small = _randn((2 * n, C), 7)
    wx[pick] = small
    x = torch.empty((rows, 64), dtype=torch.bfloat16, device="cuda")
    xs = _randn((2 * n, 64), 8)
    x[pick] = xs
    a, b = (far, counts, status), (near, counts, status)
    # long rows in: product, gradient of the weights
    assert torch.equal(M.moe_expert_gemm(wx, wide, *a)[pick], M.moe_expert_gemm(small, wide, *b))
    assert torch.equal(M.moe_expert_gemm_wgrad(x, wx, *a), M.moe_expert_gemm_wgrad(xs, small, *b))
    assert torch.equal(M.moe_expert_gemm_wgrad(wx, x, *a), M.moe_expert_gemm_wgrad(small, xs, *b))
    del wx
    # long rows out: activation, gradients of the rows
    h, gu = M.moe_expert_gemm_swiglu(x, w13, *a)
    hs, gus = M.moe_expert_gemm_swiglu(xs, w13, *b)
    assert torch.equal(h[pick], hs) and torch.equal(gu[pick], gus)
    dgu = M.moe_expert_gemm_dgrad_swiglu(x, w2, gu, *a)
    assert torch.equal(dgu[pick], M.moe_expert_gemm_dgrad_swiglu(xs, w2, gus, *b))
    assert torch.equal(M.moe_expert_gemm_dgrad(x, w2, *a)[pick], M.moe_expert_gemm_dgrad(xs, w2, *b))
    assert int(status[0]) == 0


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_past_32_bits(bits):
    n, a = 2 ** 31 + 777, 2 ** 31 - 1024
    p = torch.empty(n, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(9))
    g = torch.empty(n, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(10))
    states = [torch.zeros(n, dtype=d, device="cuda")
              for d in ((torch.int8, torch.uint8) if bits == 8 else (torch.float32, torch.float32))]
    scales = [torch.zeros(-(-n // 256), device="cuda") for _ in range(2)] if bits == 8 else []
    big = [p, g, *states, *scales]
    ends = [slice(0, 1024), slice(a, n)]   # whole blocks of 256, but for the last
    cut = [[t[e].clone() if t.numel() == n else t[e.start // 256:-(-e.stop // 256)].clone() for t in big] for e in ends]

    def step(ts):
        opt = M.moe_adamw_create(*([t] for t in ts[:4]), None, *([t] for t in ts[4:]))
        for i in (1, 2):
            M.moe_adamw_step(opt, step=i, lr=1e-2, weight_decay=0.1)

    step(big)
    for e, c in zip(ends, cut):
        step(c)
        for t, s in zip(big, c):
            part = t[e] if t.numel() == n else t[e.start // 256:-(-e.stop // 256)]
            assert torch.equal(part, s)
