"""The experts' products where their numbers are at an end: last rows that are
cleared between the two CTAs of a pair, tiles of every height, reductions that
take seconds, no rows at all.
"""

import pytest
import torch

import moe_expert_layer_ep_gb300 as M

pytestmark = pytest.mark.gpu


def _randn(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + sum(shape))
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def _at(start, counts):
    at = [torch.as_tensor(v, dtype=torch.int32, device="cuda") for v in (start, counts)]
    return (*at, torch.zeros(4, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("N,C", [(256, 256), (520, 88), (136, 640)])
def test_cleared_last_rows_are_those_of_zeros(N, C):
    """Experts of 1 to 200 rows among rows of NaN, against the same rows followed by zeros up to whole blocks of 64,
    which no clearing touches: zeros add nothing, so the same bits, call after call."""
    E, step = 200, 256
    counts = torch.arange(1, E + 1)
    dy, x = _randn(E * step, N), _randn(E * step, C)
    row = torch.arange(E * step, device="cuda")
    past = (row % step) >= (row // step + 1)
    zeros = [t.masked_fill(past[:, None], 0.0) for t in (dy, x)]
    nans = [t.masked_fill(past[:, None], float("nan")) for t in (dy, x)]
    start = torch.arange(E) * step
    want = M.moe_expert_gemm_wgrad(*zeros, *_at(start, (counts + 63) // 64 * 64))
    at = _at(start, counts)
    for _ in range(30):
        assert torch.equal(M.moe_expert_gemm_wgrad(*nans, *at), want)
    assert torch.isfinite(want).all() and int(at[2][0]) == 0


def _sparse(rows, cols, at, seed):
    """Zeros but for small whole numbers in the rows `at`: sums of their products are exact in any order."""
    t = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(seed)
    t[at] = torch.randint(-8, 9, (len(at), cols), generator=g, device="cuda").to(torch.bfloat16)
    return t


def test_weights_gradient_over_as_many_rows_as_there_may_be():
    """One expert of nearly 2^31 rows, a reduction of some 8 s: a wait for it has time enough."""
    rows = 2 ** 31 - 71
    at = torch.tensor([0, 77, 2 ** 29 + 5, rows - 58, rows - 57, rows - 1], device="cuda")
    dy, x = _sparse(rows, 8, at, 1), _sparse(rows, 8, at, 2)
    where = _at([0], [rows])
    dw = M.moe_expert_gemm_wgrad(dy, x, *where, dw=torch.empty((1, 8, 8), device="cuda"))
    assert M.moe_read_device_status(where[2]) == 0
    assert torch.equal(dw[0].double(), dy[at].double().T @ x[at].double())


def test_last_rows_after_a_long_reduction_without_any():
    """A first expert of whole blocks of 64 for some 4 s, then others whose last rows are cleared, on the same pair of
    CTAs among others."""
    E, long = 200, 2 ** 30
    rows = long + 64 * E
    start = [0] + [long + 64 * e for e in range(E - 1)]
    at = torch.tensor([3, long - 1] + [s + r for s in start[1:] for r in (0, 4)], device="cuda")
    dy, x = _sparse(rows, 8, at, 3), _sparse(rows, 8, at, 4)
    where = _at(start, [long] + [5] * (E - 1))
    dw = M.moe_expert_gemm_wgrad(dy, x, *where, dw=torch.empty((E, 8, 8), device="cuda"))
    assert M.moe_read_device_status(where[2]) == 0
    d, a = dy[at].double().view(E, 2, 8), x[at].double().view(E, 2, 8)
    assert torch.equal(dw.double(), d.transpose(1, 2) @ a)


def test_products_over_as_many_columns_as_there_may_be():
    """Reductions over nearly 2^30 columns, some 3 s each."""
    n = 2 ** 30 - 8
    at = torch.tensor([0, 1000, 2 ** 29 + 1, n - 65, n - 1], device="cuda")
    x = _sparse(n, 1, at, 5).view(1, n)
    where = _at([0], [1])
    w = _sparse(n, 8, at, 6)
    want = x[0, at].double() @ w[at].double()
    got = M.moe_expert_gemm_dgrad(x, w.view(1, n, 8), *where)
    assert M.moe_read_device_status(where[2]) == 0 and torch.equal(got[0], want.to(torch.bfloat16))
    w = w.t().contiguous().view(1, 8, n)
    got = M.moe_expert_gemm(x, w, *where)
    assert M.moe_read_device_status(where[2]) == 0 and torch.equal(got[0], want.to(torch.bfloat16))


@pytest.mark.parametrize("counts,start,fits", [([0, 0], [0, 128], True), ([0, 3], [0, 0], False), ([-1, 0], [0, 0], False)])
def test_no_sorted_rows_and_experts_that_claim_some(counts, start, fits):
    """Experts whose numbers do not fit the buffers are reported where the buffers are empty, too."""
    empty = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w, gu = _randn(2, 64, 64), torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    sums = torch.full((2, 64, 64), 7.0, device="cuda")
    for call in (lambda at: M.moe_expert_gemm(empty, w, *at), lambda at: M.moe_expert_gemm_swiglu(empty, w, *at),
                 lambda at: M.moe_expert_gemm_dgrad(empty, w, *at),
                 lambda at: M.moe_expert_gemm_dgrad_swiglu(empty, w, gu, *at),
                 lambda at: M.moe_expert_gemm_wgrad(empty, empty, *at),
                 lambda at: M.moe_expert_gemm_wgrad(empty, empty, *at, dw=sums, accumulate=True)):
        at = _at(start, counts)
        call(at)
        assert M.moe_read_device_status(at[2]) == (0 if fits else M.STATUS["MOE_ERR_INVALID_ARG"])
    assert torch.all(sums == 7.0)


def test_a_row_in_tiles_of_every_width():
    """160 experts make tiles enough that one of n rows is one MMA of n rounded up to 32 tokens wide: a row's bits are
    the same in all eight widths and in the low tiles of an expert alone, and nothing is written past an expert's
    rows."""
    E, N, C, step = 160, 144, 72, 256
    x, dy, gu = _randn(E * step, C), _randn(E * step, N), _randn(E * step, 2 * C)
    wide, w = _randn(E, 2 * N, C, seed=1), _randn(E, N, C, seed=2)
    start = torch.arange(E) * step

    def products(rows, experts, at):
        a, d, p, wa, wb = x[rows], dy[rows], gu[rows], wide[experts], w[experts]

        def out(cols):
            return torch.full((a.shape[0], cols), 7.0, dtype=torch.bfloat16, device="cuda")

        got = [M.moe_expert_gemm(a, wa, *at, y=out(2 * N)),
               *M.moe_expert_gemm_swiglu(a, wa, *at, h=out(N), gu=out(2 * N)),
               M.moe_expert_gemm_dgrad(d, wb, *at, dx=out(C)),
               M.moe_expert_gemm_dgrad_swiglu(d, wb, p, *at, dgu=out(2 * C))]
        assert int(at[2][0]) == 0
        return got

    every = slice(0, E * step)
    full = products(every, slice(0, E), _at(start, [256] * E))
    row = torch.arange(E * step, device="cuda") % step
    for n in (1, 32, 33, 64, 65, 81, 96, 97, 128, 129, 160, 161, 192, 193, 200, 224, 225, 255):
        tall = products(every, slice(0, E), _at(start, [n] * E))
        for a, b in zip(tall, full):
            assert torch.equal(a[row < n], b[row < n]) and torch.all(a[row >= n] == 7.0)
        for e in (0, 93):
            alone = products(slice(e * step, (e + 1) * step), slice(e, e + 1), _at([0], [n]))
            for a, b in zip(alone, tall):
                assert torch.equal(a, b[e * step:(e + 1) * step])
