"""The bits of products and gradients, zeros' signs among them, whichever kernel the sizes select: few tiles of 64 x 64 or
tiles of 256 features on CTA pairs, with and without a bias and a residual."""

import pytest
import torch

import moe_expert_layer_ep_gb300 as M

pytestmark = pytest.mark.gpu

ACTS = list(M.MOE_ACTS)
C, N, WIDE = 136, 72, 10_240


def _same(a, b):
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def _cut(t):
    return t[..., :N].contiguous()


def _operands(rows, seed):
    """Rows of zeros and of signed zeros among them, and weights of zeros; sums and z far below 0 too."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    x, w = rand(rows, C), rand(WIDE, C)
    x[3:rows:5] *= 30.0
    x[1:rows:7] = 0.0
    x[2:rows:7] = -0.0
    w[5:WIDE:9] = 0.0
    w[6:WIDE:9] *= -0.0
    z = rand(rows, WIDE) * 40.0
    z[:, 1:WIDE:4] = -0.0
    res = rand(rows, WIDE)
    res[:, 2:WIDE:3] = -0.0
    return [t.to(torch.bfloat16) for t in (x, w, z, res)], rand(WIDE)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows", [1, 40, 200, 700])
def test_few_tiles_and_many(rows, act):
    (x, w, z, res), b = _operands(rows, 61)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    at = (None, None, status)
    whole = [torch.tensor([v], dtype=torch.int32, device="cuda") for v in (0, rows)] + [status]   # by expert: never few tiles
    wt = w.t().contiguous()
    for bias in (None, b):
        for r in (None, res):
            for way, cols in ((at, N), (at, WIDE), (whole, N)):
                y, kept = M.moe_expert_gemm_act(x, w[:cols][None], *way, bias=None if bias is None else bias[:cols][None].contiguous(),
                                                act=act, residual=None if r is None else r[:, :cols].contiguous(), keep_z=True)
                first = (y, kept) if cols == N and way is at else first
                _same(_cut(y), first[0])
                _same(_cut(kept), first[1])
    for r in (None, res):
        for way, cols in ((at, N), (at, WIDE), (whole, N)):
            d = M.moe_expert_gemm_dgrad_act(x, wt[:, :cols].contiguous()[None], *way, z=z[:, :cols].contiguous(), act=act,
                                            residual=None if r is None else r[:, :cols].contiguous())
            first = d if cols == N and way is at else first
            _same(_cut(d), first)
    half = WIDE // 2

    def halves(t, cols):
        return torch.cat((t[..., :cols], t[..., half:half + cols]), -1).contiguous()

    for bias in (None, b):
        for way, cols in ((at, N), (at, half), (whole, N)):
            h, gu = M.moe_expert_gemm_glu(x, halves(wt, cols).t().contiguous()[None], *way,
                                          bias=None if bias is None else halves(bias, cols)[None], act=act)
            first = (h, gu) if cols == N and way is at else first
            _same(_cut(h), first[0])
            _same(torch.cat((gu[:, :N], gu[:, cols:cols + N]), 1), first[1])
    for way, cols in ((at, N), (at, half), (whole, N)):
        d = M.moe_expert_gemm_dgrad_glu(x, wt[:, :cols].contiguous()[None], halves(z, cols), *way, act=act)
        d = torch.cat((d[:, :N], d[:, cols:cols + N]), 1)
        first = d if cols == N and way is at else first
        _same(d, first)


@pytest.mark.parametrize("rows", [1, 40, 200, 700])
def test_the_plain_products(rows):
    (x, w, z, _), _ = _operands(rows, 62)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    at = (None, None, status)
    whole = [torch.tensor([v], dtype=torch.int32, device="cuda") for v in (0, rows)] + [status]
    wt = w.t().contiguous()
    for cols in (80, WIDE):
        a, d = w[:cols][None], wt[:, :cols].contiguous()[None]
        _same(M.moe_expert_gemm(x, a, *at), M.moe_expert_gemm(x, a, *whole))
        _same(M.moe_expert_gemm(x, a, *at), M.moe_expert_gemm_act(x, a, *whole)[0])
        _same(M.moe_expert_gemm_dgrad(x, d, *at), M.moe_expert_gemm_dgrad(x, d, *whole))
        for p, q in zip(M.moe_expert_gemm_swiglu(x, a, *at), M.moe_expert_gemm_glu(x, a, *whole)):
            _same(p, q)
        for p, q in zip(M.moe_expert_gemm_swiglu(x, a, *whole), M.moe_expert_gemm_glu(x, a, *at)):
            _same(p, q)
