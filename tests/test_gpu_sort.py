"""Tokens sorted by expert and back, and their gradients, against the fp64
oracle.

Tolerances: U = 2^-24 per fp32 rounding, 2^-8 relative for one rounding to
bf16.  A sum over j of k products: (k + 1) U sum|w y|.  A dot product of K
terms, in any order: K U sum|d y|.  Copies and one-term products: exact up to
their own rounding.  Rows that carry no token are filled with a pattern before
the call and have to keep it.
"""

import numpy as np
import pytest
import torch

import moe_expert_layer_ep_gb300 as M
from oracle import train as R

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
STORE = {"bf16": 2.0 ** -8, "fp32": 0.0}


def _f64(t):
    return t.detach().cpu().double().numpy()


def _ids(T, E, k, seed, drop=0.0):
    rng = np.random.default_rng(seed)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    ids[rng.random((T, k)) < drop] = -1
    return torch.from_numpy(ids)


def _randn(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(DT[dtype])


CASES = [  # T, K, E, E_local, first, topk, dtype, dropped share
    (1, 8, 4, 4, 0, 1, "bf16", 0.0), (1, 7168, 64, 64, 0, 8, "bf16", 0.0), (1, 1, 4, 4, 0, 2, "fp32", 0.0),
    (128, 256, 8, 8, 0, 2, "bf16", 0.0), (77, 1001, 40, 20, 10, 4, "fp32", 0.1), (300, 130, 16, 16, 0, 11, "bf16", 0.3),
    (65, 333, 64, 5, 59, 64, "bf16", 0.0), (500, 2048, 128, 128, 0, 8, "fp32", 0.05), (40, 64, 8, 8, 0, 3, "bf16", 1.0),
    (2050, 40, 300, 300, 0, 5, "bf16", 0.1)]


def _setup(T, K, E, El, first, k, dtype, drop):
    ids = _ids(T, E, k, T + K, drop)
    ref = R.sort_plan(ids.numpy(), E, El, first)
    rows = M.moe_compact_all_tokens(T * k, El)
    return ids, ref, rows


@pytest.mark.parametrize("case", CASES, ids=str)
def test_sort_and_back(case):
    T, K, E, El, first, k, dtype, drop = case
    ids, (dst, start, counts), rows = _setup(*case)
    ws = torch.empty(M.moe_sort_plan_workspace_size(T, k, El), dtype=torch.uint8, device="cuda")
    s2d, st, cn = M.moe_sort_plan(ids.cuda(), E, El, first, ws=ws)
    assert M.moe_read_device_status(ws) == 0
    assert np.array_equal(s2d.cpu().numpy(), dst)
    assert np.array_equal(st.cpu().numpy(), start) and np.array_equal(cn.cpu().numpy(), counts)

    x = _randn((T, K), dtype, 1)
    buf = torch.full((rows, K), 7.0, dtype=DT[dtype], device="cuda")
    out = M.moe_sort_tokens(x.cuda(), s2d, out=buf)
    assert out is buf
    assert np.array_equal(_f64(buf), R.sort_tokens(_f64(x), dst, np.full((rows, K), 7.0)))

    y = _randn((rows, K), dtype, 2)
    y[torch.from_numpy(np.setdiff1d(np.arange(rows), dst.reshape(-1)))] = float("nan")   # never read
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(3))
    y64, w64 = np.nan_to_num(_f64(y)), _f64(w)
    for weights, wq in ((None, np.ones((T, k))), (w.cuda(), w64)):
        got = _f64(M.moe_unsort_tokens(y.cuda(), s2d, weights))
        ref = R.unsort_tokens(y64, dst, wq)
        size = R.unsort_tokens(np.abs(y64), dst, np.abs(wq))
        near = (k + 1) * U * size
        assert np.all(np.abs(got - ref) <= near + STORE[dtype] * (np.abs(ref) + near))
        assert not np.any(got[np.all(dst < 0, axis=1)])

    dout = _randn((T, K), dtype, 4)
    dbuf = torch.full((rows, K), 7.0, dtype=DT[dtype], device="cuda")
    dy, dw = M.moe_unsort_tokens_backward(dout.cuda(), y.cuda(), s2d, w.cuda(), dy=dbuf)
    ref_dy, ref_dw = R.unsort_tokens_backward(_f64(dout), y64, dst, w64, np.full((rows, K), 7.0))
    assert np.all(np.abs(_f64(dy) - ref_dy) <= (U + STORE[dtype] * 1.001) * np.abs(ref_dy) * (ref_dy != 7.0))
    _, size = R.unsort_tokens_backward(np.abs(_f64(dout)), np.abs(y64), dst, w64, np.zeros((rows, K)))
    assert np.all(np.abs(_f64(dw) - ref_dw) <= K * U * size)
    assert not np.any(_f64(dw)[dst < 0])


@pytest.mark.parametrize("T,E,El,first,k", [(0, 300, 300, 0, 2), (1, 1024, 1024, 0, 1), (256, 256, 256, 0, 8),
                                            (257, 256, 256, 0, 8), (1024, 64, 64, 0, 3), (512, 8, 8, 0, 5), (70, 600, 257, 340, 64),
                                            (9000, 1024, 1000, 24, 8), (30001, 64, 32, 16, 8), (66000, 4, 4, 0, 1)])
def test_plan_of_any_size(T, E, El, first, k):
    """Every kernel of the plan (one CTA; parts of one and of several 512s), ragged ends, a status word that a call
    clears, scratch that held something else."""
    ids = _ids(T, E, k, T + E, 0.05)
    ws = torch.full((M.moe_sort_plan_workspace_size(T, k, El) + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    got = M.moe_sort_plan(ids.cuda(), E, El, first, ws=ws[:-256])
    assert M.moe_read_device_status(ws) == 0
    assert torch.all(ws[-256:] == 0xA5)
    for a, b in zip(got, R.sort_plan(ids.numpy(), E, El, first)):
        assert np.array_equal(a.cpu().numpy(), b)
    if T > 4:
        ids[3, 0], ids[T // 2, k - 1] = E, -2
        got = M.moe_sort_plan(ids.cuda(), E, El, first, ws=ws[:-256])
        assert M.moe_read_device_status(ws) == M.STATUS["MOE_ERR_EXPERT_ID"]
        for a, b in zip(got, R.sort_plan(ids.numpy(), E, El, first)):
            assert np.array_equal(a.cpu().numpy(), b)


def test_directional_derivative_of_the_weighted_way_back():
    """<dout, unsort(y, w)> is bilinear in y and w: its change along (v, z) is the gradients' product with them."""
    T, K, E, k = 60, 96, 8, 3
    ids = _ids(T, E, k, 5, 0.1).cuda()
    s2d, _, _ = M.moe_sort_plan(ids, E)
    rows = M.moe_compact_all_tokens(T * k, E)
    y, v, dout = (_randn((rows, K), "fp32", s).cuda() for s in (1, 2, 3))
    dout = dout[:T].contiguous()
    w, z = torch.rand((T, k), device="cuda"), torch.randn((T, k), device="cuda")
    dy, dw = M.moe_unsort_tokens_backward(dout, y, s2d, w, dy=torch.zeros_like(y))
    h = 0.5   # central differences of a quadratic are exact for any h

    def f(sign):
        out = M.moe_unsort_tokens(y + sign * h * v, s2d, w + sign * h * z)
        return float((out.double() * dout.double()).sum())

    slope = (f(1) - f(-1)) / (2 * h)
    grad = float((dy.double() * v.double()).sum() + (dw.double() * z.double()).sum())
    size = float(M.moe_unsort_tokens(y.abs() + v.abs(), s2d, w + z.abs()).double().mul(dout.abs().double()).sum())
    assert abs(slope - grad) <= 64 * U * size


def test_strides_alignment_and_views():
    """Rows inside wider matrices, at every offset of elements, give the bits of contiguous ones and leave the rest
    alone."""
    T, K, E, k = 33, 72, 8, 4
    s2d, _, _ = M.moe_sort_plan(_ids(T, E, k, 9).cuda(), E)
    rows = M.moe_compact_all_tokens(T * k, E)
    w = torch.rand((T, k), device="cuda")
    for dtype in DT:
        x, y = _randn((T, K), dtype, 1).cuda(), _randn((rows, K), dtype, 2).cuda()
        want = [M.moe_sort_tokens(x, s2d, out=torch.zeros_like(y)), M.moe_unsort_tokens(y, s2d, w),
                *M.moe_unsort_tokens_backward(x, y, s2d, w, dy=torch.zeros_like(y))]
        for left, width in ((0, 80), (1, 79), (3, 83), (8, 88)):
            def wide(t, fill=0.0):
                big = torch.full((t.shape[0], width), fill, dtype=t.dtype, device="cuda")
                big[:, left:left + K] = t
                return big, big[:, left:left + K]
            (_, xv), (_, yv) = wide(x), wide(y)
            big, view = wide(torch.zeros_like(y), 5.0)
            M.moe_sort_tokens(xv, s2d, out=view)
            big2, view2 = wide(torch.zeros_like(x), 5.0)
            M.moe_unsort_tokens(yv, s2d, w, out=view2)
            big3, view3 = wide(torch.zeros_like(y), 5.0)
            _, dw = M.moe_unsort_tokens_backward(xv, yv, s2d, w, dy=view3)
            assert torch.equal(view, want[0]) and torch.equal(view2, want[1]) and torch.equal(view3, want[2])
            # (another access width adds the dot products' terms in another order)
            size = float(x.abs().amax() * y.abs().amax()) * K
            assert torch.allclose(dw, want[3], rtol=0, atol=2 * K * U * size)
            for b in (big, big2, big3):
                assert torch.all(b[:, :left] == 5.0) and torch.all(b[:, left + K:] == 5.0)


def test_bad_ids_and_rows_are_dropped():
    ids = torch.tensor([[0, 9], [3, -1], [-7, 1]], dtype=torch.int32, device="cuda")
    ws = torch.empty(M.moe_sort_plan_workspace_size(3, 2, 4), dtype=torch.uint8, device="cuda")
    s2d, _, counts = M.moe_sort_plan(ids, 4, ws=ws)
    assert M.moe_read_device_status(ws) == M.STATUS["MOE_ERR_EXPERT_ID"]
    assert counts.tolist() == [1, 1, 0, 1] and s2d.tolist() == [[0, -1], [256, -1], [-1, 128]]
    # a sorted buffer that ends before some rows: those are skipped, nothing is written past it
    x = torch.randn((3, 32), device="cuda")
    guard = torch.full((260, 32), 5.0, device="cuda")
    M.moe_sort_tokens(x, s2d, out=guard[:200])
    assert torch.equal(guard[0], x[0]) and torch.equal(guard[128], x[2]) and torch.all(guard[200:] == 5.0)
    out = M.moe_unsort_tokens(guard[:200], s2d)
    assert torch.equal(out[0], x[0]) and not out[1].any()


def test_no_tokens():
    s2d, start, counts = M.moe_sort_plan(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 4)
    assert counts.tolist() == [0] * 4 and start.tolist() == [0] * 4
    x, y = torch.empty((0, 16), device="cuda"), torch.empty((128, 16), device="cuda")
    M.moe_sort_tokens(x, s2d, out=y)
    assert M.moe_unsort_tokens(y, s2d).shape == (0, 16)
    # a rank that keeps nothing and has no rows at all
    none = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    empty = torch.empty((0, 16), device="cuda")
    assert not M.moe_unsort_tokens(empty, none).any()
    _, dw = M.moe_unsort_tokens_backward(torch.ones((3, 16), device="cuda"), empty, none, torch.ones((3, 2), device="cuda"))
    assert not dw.any()


def test_same_bits_alone_in_a_batch_in_a_graph_and_on_another_stream():
    T, K, E, k = 200, 1000, 16, 4
    ids = _ids(T, E, k, 3).cuda()
    w = torch.rand((T, k), device="cuda")
    rows = M.moe_compact_all_tokens(T * k, E)
    y, dout = _randn((rows, K), "bf16", 1).cuda(), _randn((T, K), "bf16", 2).cuda()
    s2d, start, counts = M.moe_sort_plan(ids, E)
    out = M.moe_unsort_tokens(y, s2d, w)
    dy, dw = M.moe_unsort_tokens_backward(dout, y, s2d, w, dy=torch.zeros_like(y))
    for t in (0, 57, T - 1):
        one = s2d[t:t + 1].contiguous()
        assert torch.equal(M.moe_unsort_tokens(y, one, w[t:t + 1].contiguous())[0], out[t])
        _, dw1 = M.moe_unsort_tokens_backward(dout[t:t + 1], y, one, w[t:t + 1].contiguous(), dy=torch.zeros_like(y))
        assert torch.equal(dw1[0], dw[t])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [*M.moe_sort_plan(ids, E), M.moe_unsort_tokens(y, s2d, w)]
    explicit = M.moe_unsort_tokens(y, s2d, w, stream=side)
    torch.cuda.synchronize()
    for a, b in zip(got, (s2d, start, counts, out)):
        assert torch.equal(a, b)
    assert torch.equal(explicit, out)
    bufs = [torch.empty_like(t) for t in (s2d, start, counts, out)]
    ws = torch.empty(M.moe_sort_plan_workspace_size(T, k, E), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.moe_sort_plan(ids, E, src2dst=bufs[0], start=bufs[1], counts=bufs[2], ws=ws)
        M.moe_unsort_tokens(y, bufs[0], w, out=bufs[3])
    for b in bufs:
        b.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(bufs, (s2d, start, counts, out)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("K,k,dtype", [(2048, 8, "bf16"), (2048, 2, "bf16"), (1001, 8, "bf16"), (1002, 3, "bf16"),
                                       (1024, 5, "fp32"), (333, 4, "fp32")])
def test_same_bits_alone_and_among_many(K, k, dtype):
    T, E = 8000, 32
    ids = _ids(T, E, k, 21, 0.1).cuda()
    g = torch.Generator(device="cuda").manual_seed(22)
    w = torch.rand((T, k), generator=g, device="cuda")
    rows = M.moe_compact_all_tokens(T * k, E)
    y, dout = (torch.randn((n, K), generator=g, device="cuda").to(DT[dtype]) for n in (rows, T))
    s2d, _, _ = M.moe_sort_plan(ids, E)
    out = M.moe_unsort_tokens(y, s2d, w)
    dy, dw = M.moe_unsort_tokens_backward(dout, y, s2d, w, dy=torch.zeros_like(y))
    for a, b in ((0, 1), (5000, 5002), (T - 300, T)):
        some = [t[a:b].contiguous() for t in (dout, s2d, w)]
        assert torch.equal(M.moe_unsort_tokens(y, some[1], some[2]), out[a:b])
        dy1, dw1 = M.moe_unsort_tokens_backward(some[0], y, some[1], some[2], dy=torch.zeros_like(y))
        at = some[1][some[1] >= 0].long()
        assert torch.equal(dw1, dw[a:b]) and torch.equal(dy1[at], dy[at])


def _code(f):
    with pytest.raises(M.MoeError) as e:
        f()
    return M.STATUS_NAMES[e.value.code]


def test_refusals():
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    s2d, _, _ = M.moe_sort_plan(ids, 4)
    x = torch.zeros((4, 16), device="cuda")
    assert _code(lambda: M.moe_sort_plan(ids, 4, 4, 1)) == "MOE_ERR_INVALID_ARG"
    assert _code(lambda: M.moe_sort_plan(ids, 2000, 2000)) == "MOE_ERR_UNSUPPORTED"
    small = torch.empty(64, dtype=torch.uint8, device="cuda")
    assert _code(lambda: M.moe_sort_plan(ids, 4, ws=small)) == "MOE_ERR_BUFFER_TOO_SMALL"
    assert _code(lambda: M.moe_sort_tokens(torch.zeros((4, 0), device="cuda"), s2d, rows=8)) == "MOE_ERR_INVALID_ARG"
    for bad in (lambda: M.moe_sort_tokens(x.half(), s2d, rows=8), lambda: M.moe_sort_tokens(x.cpu(), s2d, rows=8),
                lambda: M.moe_sort_tokens(x.t(), s2d, rows=8), lambda: M.moe_sort_tokens(x[:3], s2d, rows=8),
                lambda: M.moe_sort_tokens(x, s2d), lambda: M.moe_sort_tokens(x, s2d, out=x.bfloat16()),
                lambda: M.moe_sort_tokens(x[:1].expand(4, 16), s2d, rows=8),
                lambda: M.moe_unsort_tokens(x, s2d, torch.ones((4, 3), device="cuda")),
                lambda: M.moe_unsort_tokens(x, s2d.long()), lambda: M.moe_sort_plan(ids.long(), 4),
                lambda: M.moe_unsort_tokens_backward(x, x[:, :8], s2d, torch.ones((4, 2), device="cuda"))):
        with pytest.raises(ValueError):
            bad()
