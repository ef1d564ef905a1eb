"""The experts' products and their gradients against the fp64 oracle.

Tolerances, on bf16 inputs: a sum of K exact products in fp32 by steps of 16 is
off by at most A = (K / 16 + 16) 2^-23 sum|a b|, and storing it in bf16 adds
2^-8 (|ref| + A).  The activation in fp32: with the exponential's
X = (4 + 1.2 |g|) 2^-23 relative error, h is off by 1.1 A_g |u| + |silu(g)| A_u
+ A_g A_u + 2 X |h|; dg by 1.1 |u| A + 4 X |dh u| s (1 + |g|), du by
|g| s A + 2 X |du|, and their storing.  Rows outside the experts hold NaN on
input and a pattern on output that has to stay.
"""

import numpy as np
import pytest
import torch

import moe_expert_layer_ep_gb300 as M
from oracle import train as R

pytestmark = pytest.mark.gpu

BF = 2.0 ** -8


def _f64(t):
    return t.detach().cpu().double().numpy()


def _randn(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


class Case:
    """Experts' rows, the gaps between them, and seeded operands."""

    def __init__(self, counts, N, C, align=128, seed=0, gap=0):
        counts = np.asarray(counts, dtype=np.int64)
        step = -(-counts // align) * align + gap
        self.counts, self.start = counts, np.concatenate([[0], np.cumsum(step)[:-1]]) + gap
        self.rows = max(1, int(step.sum()) + gap)
        self.N, self.C, self.E, self.seed = N, C, len(counts), seed
        self.valid = np.zeros(self.rows, dtype=bool)
        for s, n in zip(self.start, counts):
            self.valid[s:s + n] = True
        self.at = [torch.from_numpy(v.astype(np.int32)).cuda() for v in (self.start, counts)]
        self.at.append(torch.zeros(4, dtype=torch.int32, device="cuda"))

    def sorted(self, cols, seed, scale=1.0):
        x = _randn((self.rows, cols), self.seed + seed, scale)
        x[torch.from_numpy(~self.valid)] = float("nan")
        return x

    def weights(self, n, c, seed):
        return _randn((self.E, n, c), self.seed + seed, 1.0 / np.sqrt(c))

    def check(self, got, ref, near):
        """got: an output that was filled with 7 before; ref, near: of the valid rows."""
        got = _f64(got)
        assert np.all(got[~self.valid] == 7.0)
        v = self.valid
        assert np.all(np.abs(got[v] - ref[v]) <= near[v] + BF * (np.abs(ref[v]) + near[v]))
        assert int(self.at[2][0]) == 0

    def out(self, cols):
        return torch.full((self.rows, cols), 7.0, dtype=torch.bfloat16, device="cuda")


def _acc(K):
    return (K / 16 + 16) * 2.0 ** -23


CASES = {
    "one_row": dict(counts=[1], N=8, C=8),
    "ragged": dict(counts=[3, 0, 130, 128, 127, 1], N=136, C=72),
    "packed_rows": dict(counts=[5, 64, 0, 33, 257], N=264, C=200, align=1, gap=3),
    "middle": dict(counts=[200, 90, 16], N=512, C=768),
    "wide_columns": dict(counts=[40, 140], N=1032, C=520),
    "narrow": dict(counts=[300, 31], N=24, C=40),
    "one_tall_expert": dict(counts=[5000, 0, 7], N=256, C=320),
    "no_rows": dict(counts=[0, 0, 0], N=64, C=64),
    "many_experts": dict(counts=[i % 5 for i in range(1024)], N=64, C=128),
    "long_reduction": dict(counts=[70, 129], N=384, C=7168),
}
cases = pytest.mark.parametrize("name", CASES)


@cases
def test_forward(name):
    c = Case(**CASES[name], seed=1)
    x, w, y = c.sorted(c.C, 1), c.weights(c.N, c.C, 2), c.out(c.N)
    assert M.moe_expert_gemm(x.cuda(), w.cuda(), *c.at, y=y) is y
    x64, w64 = np.nan_to_num(_f64(x)), _f64(w)
    ref = R.expert_gemm(x64, w64, c.start, c.counts)
    c.check(y, ref, _acc(c.C) * R.expert_gemm(np.abs(x64), np.abs(w64), c.start, c.counts))


@cases
def test_forward_swiglu(name):
    c = Case(**CASES[name], seed=2)
    I = c.N
    x, w = c.sorted(c.C, 1), c.weights(2 * I, c.C, 2)
    h, gu = c.out(I), c.out(2 * I)
    M.moe_expert_gemm_swiglu(x.cuda(), w.cuda(), *c.at, h=h, gu=gu)
    x64, w64 = np.nan_to_num(_f64(x)), _f64(w)
    ref = R.expert_gemm(x64, w64, c.start, c.counts)
    near = _acc(c.C) * R.expert_gemm(np.abs(x64), np.abs(w64), c.start, c.counts)
    c.check(gu, ref, near)
    g, u = np.split(ref, 2, axis=1)
    ag, au = np.split(near, 2, axis=1)
    silu, X = g / (1 + np.exp(-g)), (4 + 1.2 * np.abs(g)) * 2.0 ** -23
    c.check(h, silu * u, 1.1 * ag * np.abs(u) + np.abs(silu) * au + ag * au + 2 * X * np.abs(silu * u))
    # without the stored halves: the same h
    h2 = c.out(I)
    _, none = M.moe_expert_gemm_swiglu(x.cuda(), w.cuda(), *c.at, h=h2, keep_gu=False)
    assert none is None and torch.equal(h, h2)


@cases
def test_dgrad(name):
    c = Case(**CASES[name], seed=3)
    dy, w, dx = c.sorted(c.N, 1), c.weights(c.N, c.C, 2), c.out(c.C)
    M.moe_expert_gemm_dgrad(dy.cuda(), w.cuda(), *c.at, dx=dx)
    d64, w64 = np.nan_to_num(_f64(dy)), _f64(w)
    ref = R.expert_gemm_dgrad(d64, w64, c.start, c.counts)
    c.check(dx, ref, _acc(c.N) * R.expert_gemm_dgrad(np.abs(d64), np.abs(w64), c.start, c.counts))


@cases
def test_dgrad_swiglu(name):
    c = Case(**CASES[name], seed=4)
    I = c.C
    dy, w, gu, dgu = c.sorted(c.N, 1), c.weights(c.N, I, 2), c.sorted(2 * I, 3, 2.0), c.out(2 * I)
    M.moe_expert_gemm_dgrad_swiglu(dy.cuda(), w.cuda(), gu.cuda(), *c.at, dgu=dgu)
    d64, w64, gu64 = np.nan_to_num(_f64(dy)), _f64(w), np.nan_to_num(_f64(gu))
    dh = R.expert_gemm_dgrad(d64, w64, c.start, c.counts)
    A = _acc(c.N) * R.expert_gemm_dgrad(np.abs(d64), np.abs(w64), c.start, c.counts)
    ref = R.swiglu_backward(dh, gu64)
    g, u = np.split(gu64, 2, axis=1)
    s, X = 1 / (1 + np.exp(-g)), (4 + 1.2 * np.abs(g)) * 2.0 ** -23
    near = np.concatenate([1.1 * np.abs(u) * A + 4 * X * np.abs(dh * u) * s * (1 + np.abs(g)),
                           np.abs(g) * s * A + 2 * X * np.abs(dh * g * s)], axis=1)
    c.check(dgu, ref, near)


@cases
def test_wgrad(name):
    c = Case(**CASES[name], seed=5)
    dy, x = c.sorted(c.N, 1), c.sorted(c.C, 2)
    dw = torch.full((c.E, c.N, c.C), 7.0, dtype=torch.bfloat16, device="cuda")
    M.moe_expert_gemm_wgrad(dy.cuda(), x.cuda(), *c.at, dw=dw)
    d64, x64 = np.nan_to_num(_f64(dy)), np.nan_to_num(_f64(x))
    ref = R.expert_gemm_wgrad(d64, x64, c.start, c.counts)
    size = R.expert_gemm_wgrad(np.abs(d64), np.abs(x64), c.start, c.counts)
    near = (c.counts / 16 + 16)[:, None, None] * 2.0 ** -23 * size
    assert np.all(np.abs(_f64(dw) - ref) <= near + BF * (np.abs(ref) + near))
    assert int(c.at[2][0]) == 0


@cases
def test_wgrad_in_fp32_stored_and_added(name):
    """The unrounded sums: within their bound, the bf16 output before its rounding; added to what dw holds with one
    rounding to fp32, which is the sum that torch forms.  Nothing around dw is written."""
    c = Case(**CASES[name], seed=15)
    dy, x = c.sorted(c.N, 1), c.sorted(c.C, 2)
    d64, x64 = np.nan_to_num(_f64(dy)), np.nan_to_num(_f64(x))
    dy, x = dy.cuda(), x.cuda()
    size = c.E * c.N * c.C
    around = torch.full((size + 64,), 5.0, device="cuda")
    dw = around[32:32 + size].view(c.E, c.N, c.C)
    M.moe_expert_gemm_wgrad(dy, x, *c.at, dw=dw)
    ref = R.expert_gemm_wgrad(d64, x64, c.start, c.counts)
    near = (c.counts / 16 + 16)[:, None, None] * 2.0 ** -23 * R.expert_gemm_wgrad(np.abs(d64), np.abs(x64), c.start,
                                                                                  c.counts)
    assert np.all(np.abs(_f64(dw) - ref) <= near)
    assert torch.equal(dw.to(torch.bfloat16), M.moe_expert_gemm_wgrad(dy, x, *c.at))
    one = dw.clone()
    base = torch.randn((c.E, c.N, c.C), generator=torch.Generator().manual_seed(16)).cuda()
    dw.copy_(base)
    for _ in range(3):
        M.moe_expert_gemm_wgrad(dy, x, *c.at, dw=dw, accumulate=True)
        base = base + one
        assert torch.equal(dw, base)
    assert torch.all(around[:32] == 5.0) and torch.all(around[32 + size:] == 5.0)
    assert int(c.at[2][0]) == 0


def test_wgrad_in_fp32_refusals_and_no_rows():
    c = Case([4], N=64, C=64)
    x = torch.zeros((128, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(M.MoeError) as e:
        M.moe_expert_gemm_wgrad(x, x, *c.at, dw=torch.zeros((1, 64, 64), device="cuda").bfloat16(), accumulate=True)
    assert M.STATUS_NAMES[e.value.code] == "MOE_ERR_UNSUPPORTED"
    with pytest.raises(M.MoeError) as e:
        M.moe_expert_gemm_wgrad(x, x, *c.at, dw=torch.zeros(64 * 64 + 1, device="cuda")[1:].view(1, 64, 64))
    assert M.STATUS_NAMES[e.value.code] == "MOE_ERR_MISALIGNED"
    for bad in (dict(accumulate=True), dict(dw=torch.zeros((1, 64, 64), dtype=torch.float64, device="cuda")),
                dict(dw=torch.zeros((1, 64, 32), device="cuda")), dict(dw=torch.zeros((1, 64, 128), device="cuda")[..., ::2])):
        with pytest.raises(ValueError):
            M.moe_expert_gemm_wgrad(x, x, *c.at, **bad)
    empty, dw = x[:0], torch.full((1, 64, 64), 7.0, device="cuda")
    assert torch.all(M.moe_expert_gemm_wgrad(empty, empty, *c.at, dw=dw, accumulate=True) == 7.0)
    assert not M.moe_expert_gemm_wgrad(empty, empty, *c.at, dw=dw).any()


def test_gradients_are_those_of_the_forward_product():
    """sum(dy * y) is linear in x and in w, so it equals sum(dx * x) and sum(dw * w): the stored outputs' rounding is
    the difference, at most 2^-8 of the terms' sizes."""
    c = Case([100, 0, 260, 5], N=160, C=96, seed=6)
    x, dy = (torch.nan_to_num(c.sorted(n, s)).cuda() for n, s in ((c.C, 1), (c.N, 2)))
    w = c.weights(c.N, c.C, 3).cuda()
    zero = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    y = M.moe_expert_gemm(x, w, *c.at, y=zero(c.rows, c.N)).double()
    dx = M.moe_expert_gemm_dgrad(dy, w, *c.at, dx=zero(c.rows, c.C)).double()
    dw = M.moe_expert_gemm_wgrad(dy, x, *c.at).double()
    pairs = [(dy.double(), y), (dx, x.double()), (dw, w.double())]
    sums = [float((a * b).sum()) for a, b in pairs]
    size = max(float((a * b).abs().sum()) for a, b in pairs)
    assert max(sums) - min(sums) <= 2 * (BF + _acc(260)) * size


def test_differences_through_the_activation():
    """The loss sum(dh * h) along a direction of x: differences of stored h (in bf16) against the gradient."""
    c = Case([60, 0, 150], N=64, C=128, seed=7)
    x, v = (torch.nan_to_num(c.sorted(c.C, s)).cuda() for s in (1, 2))
    w13 = c.weights(2 * c.N, c.C, 3).cuda()
    w2 = c.weights(c.C, c.N, 4).cuda()     # dh = dy W2
    dy = torch.nan_to_num(c.sorted(c.C, 5)).cuda()
    zero = lambda n: torch.zeros((c.rows, n), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    _, gu = M.moe_expert_gemm_swiglu(x, w13, *c.at, h=zero(c.N), gu=zero(2 * c.N))
    dgu = M.moe_expert_gemm_dgrad_swiglu(dy, w2, gu, *c.at, dgu=zero(2 * c.N))
    dx = M.moe_expert_gemm_dgrad(dgu, w13, *c.at, dx=zero(c.C)).double()
    dh = np.nan_to_num(R.expert_gemm_dgrad(_f64(dy), _f64(w2), c.start, c.counts))

    def loss(a):
        g = R.expert_gemm(a, _f64(w13), c.start, c.counts)
        return float(np.nansum(R.swiglu(g) * dh))

    x64, v64, t = _f64(x), _f64(v), 1e-4
    slope = (loss(x64 + t * v64) - loss(x64 - t * v64)) / (2 * t)
    grad = float((dx * v.double()).sum())
    # gu, dgu and dx were each rounded to bf16 once: their effects add up over the terms of the sum
    size = float((dx.abs() * v.double().abs()).sum())
    assert abs(slope - grad) <= 4 * BF * size


def test_rows_do_not_depend_on_the_others():
    c = Case([300, 40, 128], N=320, C=256, seed=8)
    x, w = torch.nan_to_num(c.sorted(c.C, 1)).cuda(), c.weights(c.N, c.C, 2).cuda()
    gu = torch.nan_to_num(c.sorted(2 * c.C, 4)).cuda()
    dy = torch.nan_to_num(c.sorted(c.N, 3)).cuda()

    def all_rows(start, counts, rows):
        at = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in (start, counts)] + [c.at[2]]
        xs, ds, gs = x[rows].contiguous(), dy[rows].contiguous(), gu[rows].contiguous()
        return [M.moe_expert_gemm(xs, w, *at), *M.moe_expert_gemm_swiglu(xs, w, *at),
                M.moe_expert_gemm_dgrad(ds, w, *at), M.moe_expert_gemm_dgrad_swiglu(ds, w, gs, *at)]

    full = all_rows(c.start.tolist(), c.counts.tolist(), torch.arange(c.rows, device="cuda"))
    some = torch.tensor([7, 290, int(c.start[1]) + 3, int(c.start[2]) + 100], device="cuda")
    for a, b in zip(all_rows([0, 2, 3], [2, 1, 1], some), full):
        assert torch.equal(a, b[some])


def test_a_row_at_every_tile_height():
    """The same row first among 1 to 300 others, so in MMAs of every width: the same bits."""
    N, C = 144, 200
    g = torch.Generator().manual_seed(11)
    x = torch.randn((300, C), generator=g).to(torch.bfloat16).cuda()
    dy = torch.randn((300, N), generator=g).to(torch.bfloat16).cuda()
    gu = torch.randn((300, 2 * C), generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn((1, N, C), generator=g) * 0.1).to(torch.bfloat16).cuda()
    first = None
    for n in (1, 32, 33, 64, 65, 97, 128, 129, 161, 193, 225, 255, 256, 257, 289, 300):
        at = [torch.tensor([v], dtype=torch.int32, device="cuda") for v in (0, n)]
        at.append(torch.zeros(4, dtype=torch.int32, device="cuda"))
        got = [M.moe_expert_gemm(x[:n], w, *at), *M.moe_expert_gemm_swiglu(x[:n], w, *at),
               M.moe_expert_gemm_dgrad(dy[:n], w, *at), M.moe_expert_gemm_dgrad_swiglu(dy[:n], w, gu[:n], *at)]
        first = first or [t[0].clone() for t in got]
        for a, b in zip(got, first):
            assert torch.equal(a[0], b)


def test_tall_tiles_and_low_ones_agree():
    """160 experts of n rows make tiles enough to take them 256 rows at a time, one expert alone is cut lower: every
    row the same bits, and nothing written past an expert's rows."""
    E, N, C, step = 160, 144, 72, 304
    g = torch.Generator(device="cuda").manual_seed(17)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    x, dy, gu, w, w2 = rand(E * step, C), rand(E * step, N), rand(E * step, 2 * C), rand(E, 2 * N, C), rand(E, N, C)
    start = torch.arange(E, dtype=torch.int32, device="cuda") * step
    for n in (1, 31, 64, 97, 130, 192, 225, 256, 257, 300):
        at = [start, torch.full_like(start, n), torch.zeros(4, dtype=torch.int32, device="cuda")]

        def out(rows, cols):
            return torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device="cuda")

        def products(a, d, p, wa, wb, where, rows):
            return [M.moe_expert_gemm(a, wa, *where, y=out(rows, 2 * N)),
                    *M.moe_expert_gemm_swiglu(a, wa, *where, h=out(rows, N), gu=out(rows, 2 * N)),
                    M.moe_expert_gemm_dgrad(d, wb, *where, dx=out(rows, C)),
                    M.moe_expert_gemm_dgrad_swiglu(d, wb, p, *where, dgu=out(rows, 2 * C))]

        tall = products(x, dy, gu, w, w2, at, E * step)
        assert int(at[2][0]) == 0
        for e in (0, 77, 159):
            rows = slice(e * step, (e + 1) * step)
            one = [torch.zeros(1, dtype=torch.int32, device="cuda"), at[1][:1], at[2]]
            low = products(x[rows], dy[rows], gu[rows], w[e:e + 1], w2[e:e + 1], one, step)
            for a, b in zip(tall, low):
                assert torch.equal(a[rows], b)
                assert torch.all(b[n:] == 7.0) and torch.isfinite(b[:n]).all()


def test_weights_gradient_of_every_number_of_rows():
    """0 to 131 rows: every length of the last block of 64, next to rows that hold NaN."""
    c = Case(list(range(132)), N=40, C=24, align=8, seed=12, gap=1)
    dy, x = c.sorted(c.N, 1), c.sorted(c.C, 2)
    dw = M.moe_expert_gemm_wgrad(dy.cuda(), x.cuda(), *c.at)
    d64, x64 = np.nan_to_num(_f64(dy)), np.nan_to_num(_f64(x))
    ref = R.expert_gemm_wgrad(d64, x64, c.start, c.counts)
    size = R.expert_gemm_wgrad(np.abs(d64), np.abs(x64), c.start, c.counts)
    near = (c.counts / 16 + 16)[:, None, None] * 2.0 ** -23 * size
    assert np.all(np.abs(_f64(dw) - ref) <= near + BF * (np.abs(ref) + near))


def test_full_size_sampled():
    """A wide layer (16 experts of 7168 x 2048, 200 to 700 rows each): all outputs finite, sampled rows, and sampled
    rows of a sampled expert's dW, against fp64."""
    rng = np.random.default_rng(13)
    counts = rng.integers(200, 700, 16)
    counts[5] = 0
    start = np.concatenate([[0], np.cumsum(-(-counts // 128) * 128)[:-1]])
    rows, N, C = int(start[-1] + 768), 7168, 2048
    at = [torch.from_numpy(v.astype(np.int32)).cuda() for v in (start, counts)]
    at.append(torch.zeros(4, dtype=torch.int32, device="cuda"))
    g = torch.Generator(device="cuda").manual_seed(14)
    x, dy = (torch.randn((rows, n), generator=g, device="cuda").to(torch.bfloat16) for n in (C, N))
    w = (torch.randn((16, N, C), generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    y, dx = M.moe_expert_gemm(x, w, *at), M.moe_expert_gemm_dgrad(dy, w, *at)
    dw = M.moe_expert_gemm_wgrad(dy, x, *at)
    assert int(at[2][0]) == 0 and torch.isfinite(dw).all() and not dw[5].any()
    for e in (0, 4, 15):
        a, b, we = int(start[e]), int(start[e] + counts[e]), w[e].double()
        assert torch.isfinite(y[a:b]).all() and torch.isfinite(dx[a:b]).all()
        for r in (a, (a + b) // 2, b - 1):
            for got, v, m, K in ((y[r], x[r].double(), we.T, C), (dx[r], dy[r].double(), we, N)):
                ref, near = v @ m, _acc(K) * (v.abs() @ m.abs())
                assert torch.all((got.double() - ref).abs() <= near + BF * (ref.abs() + near))
        for n in (0, 255, 256, 4099, N - 1):
            d, xe = dy[a:b, n].double(), x[a:b].double()
            ref, near = d @ xe, _acc(counts[e]) * (d.abs() @ xe.abs())
            assert torch.all((dw[e, n].double() - ref).abs() <= near + BF * (ref.abs() + near))


def test_strides_graph_and_stream():
    c = Case([70, 0, 129], N=136, C=72, seed=9)
    x, dy = torch.nan_to_num(c.sorted(c.C, 1)).cuda(), torch.nan_to_num(c.sorted(c.N, 2)).cuda()
    w = c.weights(c.N, c.C, 3).cuda()

    def wide(t):
        big = torch.full((t.shape[0], t.shape[1] + 24), 5.0, dtype=t.dtype, device="cuda")
        big[:, 8:8 + t.shape[1]] = t
        return big, big[:, 8:8 + t.shape[1]]

    y = M.moe_expert_gemm(x, w, *c.at, y=c.out(c.N))
    dw = M.moe_expert_gemm_wgrad(dy, x, *c.at)
    _, xv = wide(x)
    _, dv = wide(dy)
    big, yv = wide(c.out(c.N))
    M.moe_expert_gemm(xv, w, *c.at, y=yv)
    assert torch.equal(yv, y) and torch.all(big[:, :8] == 5.0) and torch.all(big[:, -16:] == 5.0)
    assert torch.equal(M.moe_expert_gemm_wgrad(dv, xv, *c.at), dw)
    y2, dw2 = c.out(c.N), torch.zeros_like(dw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.moe_expert_gemm(x, w, *c.at, y=y2)
        M.moe_expert_gemm_wgrad(dy, x, *c.at, dw=dw2)
    y2.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y2, y) and torch.equal(dw2, dw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y3 = M.moe_expert_gemm(x, w, *c.at, y=c.out(c.N), stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y3, y)


def test_numbers_that_do_not_fit_are_left_out():
    c = Case([64, 32], N=64, C=64, seed=10)
    x, w = torch.nan_to_num(c.sorted(c.C, 1)).cuda(), c.weights(c.N, c.C, 2).cuda()
    want = M.moe_expert_gemm(x, w, *c.at, y=c.out(c.N))
    for start, counts in (([0, c.rows - 31], [64, 32]), ([0, -1], [64, 32]), ([0, 128], [64, -5]),
                          ([0, 128], [64, 2 ** 31 - 1])):
        at = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in (start, counts)]
        status = torch.zeros(4, dtype=torch.int32, device="cuda")
        y = M.moe_expert_gemm(x, w, *at, status, y=c.out(c.N))
        dw = M.moe_expert_gemm_wgrad(x, x, *at, status)
        assert M.moe_read_device_status(status) == M.STATUS["MOE_ERR_INVALID_ARG"]
        assert torch.equal(y[:64], want[:64]) and torch.all(y[64:] == 7.0)
        assert not dw[1].any() and dw[0].any()


def test_no_sorted_rows():
    at = [torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"),
          torch.zeros(4, dtype=torch.int32, device="cuda")]
    empty, w = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), torch.ones((2, 64, 64), device="cuda").bfloat16()
    assert M.moe_expert_gemm(empty, w, *at).shape == (0, 64)
    dw = torch.full((2, 64, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    assert not M.moe_expert_gemm_wgrad(empty, empty, *at, dw=dw).any()


def test_refusals():
    c = Case([4], N=64, C=64)
    x, w = torch.zeros((128, 64), dtype=torch.bfloat16, device="cuda"), c.weights(64, 64, 1).cuda()

    def code(f):
        with pytest.raises(M.MoeError) as e:
            f()
        return M.STATUS_NAMES[e.value.code]

    odd = torch.zeros((1, 64, 60), dtype=torch.bfloat16, device="cuda")
    assert code(lambda: M.moe_expert_gemm(x[:, :60], odd, *c.at)) == "MOE_ERR_UNSUPPORTED"
    shifted = torch.zeros((128, 72), dtype=torch.bfloat16, device="cuda")[:, 4:68]
    assert code(lambda: M.moe_expert_gemm(shifted, w, *c.at)) == "MOE_ERR_MISALIGNED"
    assert code(lambda: M.moe_expert_gemm(torch.zeros((128, 68), device="cuda").bfloat16()[:, :64], w, *c.at)) == \
        "MOE_ERR_UNSUPPORTED"
    big = torch.zeros(1025, dtype=torch.int32, device="cuda")
    assert code(lambda: M.moe_expert_gemm(x[:, :8], torch.zeros((1025, 8, 8), device="cuda").bfloat16(), big, big,
                                          c.at[2])) == "MOE_ERR_UNSUPPORTED"
    for bad in (lambda: M.moe_expert_gemm(x.float(), w, *c.at), lambda: M.moe_expert_gemm(x, w.float(), *c.at),
                lambda: M.moe_expert_gemm(x[:, :32], w, *c.at), lambda: M.moe_expert_gemm(x, w[0], *c.at),
                lambda: M.moe_expert_gemm(x, w, c.at[0].long(), *c.at[1:]),
                lambda: M.moe_expert_gemm(x, w, *c.at[:2], torch.zeros(4)),
                lambda: M.moe_expert_gemm(x, w, *c.at, y=x[:64]), lambda: M.moe_expert_gemm_wgrad(x, x[:64], *c.at),
                lambda: M.moe_expert_gemm_dgrad_swiglu(x, w, x, *c.at),
                lambda: M.moe_expert_gemm_swiglu(x, torch.zeros((1, 9, 64), device="cuda").bfloat16(), *c.at)):
        with pytest.raises(ValueError):
            bad()
