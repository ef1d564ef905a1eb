"""One AdamW step over many tensors against the fp64 oracle.

Tolerances, U = 2^-24 per fp32 rounding: with M = beta1 |m| + (1 - beta1) |g'|,
m is off by at most 5 U M (constants, products, scaled gradient, sum) and v
relatively by 6 U; the step lr' M / denom relatively by 16 U more at most, p by
4 U |p| + 16 U lr' M / denom, and 2^-8 |p| where it is stored as bf16.  States
that came in as codes add 5 U to m's and v's.  8-bit codes are the nearest to
the oracle's unrounded ones: 1/2 plus what the error e of the value's share
moves its root by, min(sqrt(e), e / sqrt(share)), times the code's range.
"""

import numpy as np
import pytest
import torch

import moe_expert_layer_ep_gb300 as M
from oracle import train as R

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HYPER = dict(step=7, lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)


def _f64(t):
    return t.detach().cpu().double().numpy()


def _at(values, dtype, offset=0):
    """values on the device, `offset` elements into their storage."""
    buf = torch.empty(values.numel() + offset, dtype=dtype, device="cuda")
    buf[offset:] = values.to(dtype)
    return buf[offset:]


class Tensor:
    def __init__(self, n, param, grad, bits, master, seed, offset=0, zero=False):
        g = torch.Generator().manual_seed(seed)
        self.n, self.bits = n, bits
        full = torch.randn(n, generator=g) * 0.1
        self.p = _at(full, DT[param], offset)
        self.w = _at(full, torch.float32, offset) if master else None
        grads = torch.randn(n, generator=g) * torch.exp2(torch.randint(-12, 3, (n,), generator=g).float())
        self.g = _at(grads * (0.0 if zero else 1.0), DT[grad], offset)
        m, v = torch.randn(n, generator=g) * 0.3, torch.randn(n, generator=g).pow(4)
        if zero:
            m, v = torch.zeros(n), torch.zeros(n)
        self.ms = self.vs = None
        if bits == 32:
            self.m, self.v = _at(m, torch.float32, offset), _at(v, torch.float32, offset)
        else:
            m, v = m.double().numpy(), v.double().numpy()
            sm, sv = R.state_scales(m).astype(np.float32), R.state_scales(v).astype(np.float32)
            cm = np.clip(np.round(R.state_roots(m, 2, 127, sm)), -127, 127)
            cv = np.clip(np.round(R.state_roots(v, 4, 255, sv)), 0, 255)
            self.m = _at(torch.from_numpy(cm), torch.int8, offset)
            self.v = _at(torch.from_numpy(cv), torch.uint8, offset)
            self.ms, self.vs = torch.from_numpy(sm).cuda(), torch.from_numpy(sv).cuda()

    def clone(self):
        c = object.__new__(Tensor)
        c.n, c.bits = self.n, self.bits
        for k in ("p", "w", "g", "m", "v", "ms", "vs"):
            t = getattr(self, k)
            setattr(c, k, None if t is None else t.clone())
        return c

    def all(self):
        return [t for t in (self.p, self.w, self.m, self.v, self.ms, self.vs) if t is not None]

    def state64(self):
        if self.bits == 32:
            return _f64(self.m), _f64(self.v)
        return (R.state_values(_f64(self.m), 2, 127, _f64(self.ms)), R.state_values(_f64(self.v), 4, 255, _f64(self.vs)))

    def want(self, scale=1.0, **hyper):
        m, v = self.state64()
        return R.adamw(_f64(self.p if self.w is None else self.w), _f64(self.g), m, v, grad_scale=scale, **hyper)


def _create(ts):
    some = lambda k: [getattr(t, k) for t in ts]  # noqa: E731
    return M.moe_adamw_create(some("p"), some("g"), some("m"), some("v"), masters=some("w"), avg_scales=some("ms"),
                              sq_scales=some("vs"))


def _check(before, after, scale=1.0, **hyper):
    m0, v0 = before.state64()
    p, m, v = before.want(scale, **hyper)
    coded = before.bits == 8
    g = np.abs(_f64(before.g) * scale)
    size = hyper["beta1"] * np.abs(m0) + (1 - hyper["beta1"]) * g
    em, ev = (10 if coded else 5) * U * size, (11 if coded else 6) * U * v
    denom = np.sqrt(v / (1 - hyper["beta2"] ** hyper["step"])) + hyper["eps"]
    step = hyper["lr"] / (1 - hyper["beta1"] ** hyper["step"]) * size / denom
    ep = 4 * U * np.abs(_f64(before.p)) * 1.01 + 20 * U * step
    if after.w is not None:
        assert np.all(np.abs(_f64(after.w) - p) <= ep)
        assert torch.equal(after.p, after.w.to(torch.bfloat16))
    else:
        store = 2.0 ** -8 * (np.abs(p) + ep) if after.p.dtype == torch.bfloat16 else 0.0
        assert np.all(np.abs(_f64(after.p) - p) <= ep + store)
    if not coded:
        assert np.all(np.abs(_f64(after.m) - m) <= em) and np.all(np.abs(_f64(after.v) - v) <= ev)
        return
    for k, x, e, power, levels in (("m", m, em, 2, 127), ("v", v, ev, 4, 255)):
        codes, scales, top = _f64(getattr(after, k)), _f64(getattr(after, k + "s")), R.state_scales(x)
        worst = R.state_scales(e)
        assert np.all(np.abs(scales - top) <= worst + U * top)
        per = np.repeat(top, R.STATE_BLOCK)[: x.size]
        share = np.divide(np.abs(x), per, out=np.zeros_like(x), where=per > 0)
        es = np.divide(e + np.repeat(worst, R.STATE_BLOCK)[: x.size] * share, per, out=np.zeros_like(x), where=per > 0)
        root = share ** 0.5
        move = np.minimum(np.sqrt(es), es / np.maximum(root, 1e-300))
        if k == "v":
            move = np.divide(move, np.sqrt(np.maximum(root, 1e-300)))
        slack = 0.5 + levels * (move + 8 * U)
        off = np.abs(codes - R.state_roots(x, power, levels, top))
        assert np.all((off <= slack) | ((k == "v") & (codes == 1) & (x > 0)))
        assert k == "m" or np.all(codes[x > 0] >= 1)


SIZES = [1, 3, 255, 256, 257, 2047, 2048, 4099, 70001]


@pytest.mark.parametrize("param,grad,master", [("fp32", "fp32", False), ("fp32", "bf16", False), ("bf16", "bf16", False),
                                               ("bf16", "fp32", False), ("bf16", "bf16", True), ("bf16", "fp32", True)])
@pytest.mark.parametrize("bits", [32, 8])
def test_step_matches_oracle(param, grad, master, bits):
    ts = [Tensor(n, param, grad, bits, master, n, offset=i % 3) for i, n in enumerate(SIZES)]
    before = [t.clone() for t in ts]
    scale = torch.tensor([0.37], device="cuda")
    opt = _create(ts)
    assert M.moe_adamw_launches(opt) == 1
    M.moe_adamw_step(opt, grad_scale=scale, **HYPER)
    torch.cuda.synchronize()
    for b, a in zip(before, ts):
        _check(b, a, float(scale.double()), **HYPER)


def test_large_tensors_take_longer_chunks():
    ts = [Tensor(n, "bf16", "bf16", 8, True, n) for n in (5_000_001, 8191, 4_000_000)]
    before = [t.clone() for t in ts]
    M.moe_adamw_step(_create(ts), **HYPER)
    torch.cuda.synchronize()
    for b, a in zip(before, ts):
        _check(b, a, **HYPER)


def test_many_tensors_of_mixed_types_are_those_stepped_alone():
    kinds = [("fp32", "fp32", 32, False), ("bf16", "bf16", 8, True), ("bf16", "fp32", 32, True), ("fp32", "bf16", 8, False)]
    ts = [Tensor(1 + 37 * i % 900, *kinds[i % 4 if i % 7 else 0], seed=i, offset=i % 2) for i in range(1000)]
    alone = [t.clone() for t in ts]
    opt = _create(ts)
    assert 4 <= M.moe_adamw_launches(opt) <= 8
    M.moe_adamw_step(opt, **HYPER)
    for t in alone[::19]:
        M.moe_adamw_step(_create([t]), **HYPER)
    torch.cuda.synchronize()
    for a, b in list(zip(ts, alone))[::19]:
        for x, y in zip(a.all(), b.all()):
            assert torch.equal(x, y)


def test_several_steps_from_nothing():
    """From zero states, five steps in 32 bits stay on the oracle's, with an error that grows by a step's each time."""
    t = Tensor(3001, "fp32", "fp32", 32, False, 1, zero=True)
    opt = _create([t])
    p, m, v = (_f64(x) for x in (t.p, t.m, t.v))
    for step in range(1, 6):
        t.g.copy_(torch.randn(3001, generator=torch.Generator().manual_seed(step)))
        h = dict(HYPER, step=step)
        M.moe_adamw_step(opt, **h)
        p, m, v = R.adamw(p, _f64(t.g), m, v, **h)
        torch.cuda.synchronize()
        # |m| <= max |g| < 5 throughout and the step is at most lr * 10
        assert np.max(np.abs(_f64(t.m) - m)) <= step * 5 * U * 5
        assert np.max(np.abs(_f64(t.p) - p)) <= step * (4 * U * 0.6 + 20 * U * h["lr"] * 10 * 5)


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_gradients_and_states(bits):
    t = Tensor(700, "fp32", "fp32", bits, False, 5, zero=True)
    before = t.clone()
    M.moe_adamw_step(_create([t]), **HYPER)
    torch.cuda.synchronize()
    want = _f64(before.p) * (1 - HYPER["lr"] * HYPER["weight_decay"])
    assert np.all(np.abs(_f64(t.p) - want) <= 2 * U * np.abs(want))
    for x in t.all()[1:]:
        assert not x.any()


def test_tiny_and_huge_second_moments_in_8_bits():
    """v > 0 keeps a code whatever its share of the block; subnormal and large scales stay finite."""
    for scale in (1e-21, 1e-16, 1.0, 1e15):
        t = Tensor(512, "fp32", "fp32", 8, False, 6, zero=True)
        g = torch.ones(512)
        g[1:256] = 1e-7
        t.g.copy_(g * scale)
        M.moe_adamw_step(_create([t]), **dict(HYPER, step=1))
        torch.cuda.synchronize()
        v = (_f64(t.g) ** 2 * (1 - HYPER["beta2"])).astype(np.float32)
        assert torch.all(t.v.cpu()[torch.from_numpy(v > 0)] >= 1)
        for x in t.all():
            assert torch.isfinite(x.float()).all()


def test_a_gradient_that_is_not_finite_is_seen():
    t = Tensor(600, "fp32", "fp32", 8, False, 7)
    t.g[300] = float("nan")
    M.moe_adamw_step(_create([t]), **HYPER)
    torch.cuda.synchronize()
    bad = ~torch.isfinite(t.p.cpu())
    assert bad.nonzero().flatten().tolist() == [300]
    assert torch.isnan(t.ms.cpu()).tolist() == [False, True, False]


def test_graph_and_stream():
    t = Tensor(5000, "bf16", "bf16", 8, True, 8)
    other, third = t.clone(), t.clone()
    M.moe_adamw_step(_create([t]), **HYPER)
    opt = _create([other])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    M.moe_adamw_step(opt, stream=side, **HYPER)
    opt3 = _create([third])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.moe_adamw_step(opt3, **HYPER)
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(t.all(), other.all(), third.all()):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_refusals():
    def code(f):
        with pytest.raises(M.MoeError) as e:
            f()
        return M.STATUS_NAMES[e.value.code]

    t = Tensor(100, "bf16", "bf16", 8, True, 9)
    opt = _create([t])
    for bad in (dict(step=0), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=float("nan")), dict(lr=float("inf"))):
        assert code(lambda: M.moe_adamw_step(opt, **dict(HYPER, **bad))) == "MOE_ERR_INVALID_ARG"
    f = Tensor(100, "fp32", "fp32", 32, False, 9)
    lists = [[f.p], [f.g], [f.m], [f.v]]
    assert code(lambda: M.moe_adamw_create(*lists, masters=[f.m])) == "MOE_ERR_DTYPE_MISMATCH"
    assert code(lambda: M.moe_adamw_create(*lists, avg_scales=[t.ms], sq_scales=[t.vs])) == "MOE_ERR_DTYPE_MISMATCH"
    assert code(lambda: M.moe_adamw_create([t.p], [t.g], [t.m], [t.v])) == "MOE_ERR_DTYPE_MISMATCH"
    for args in ([[f.p], [f.g, f.g], [f.m], [f.v]], [[f.p], [f.g[:50]], [f.m], [f.v]], [[f.p.half()], [f.g], [f.m], [f.v]],
                 [[f.p.cpu()], [f.g], [f.m], [f.v]], [[f.p], [f.g], [f.m], [t.v]]):
        with pytest.raises(ValueError):
            M.moe_adamw_create(*args)
    assert M.moe_adamw_launches(M.moe_adamw_create([], [], [], [])) == 0
