"""The operators of one training step of the expert layer, as cases to measure.

Three operators, each in its forward and backward directions:

  sort     tokens sorted by expert and back: the plan and the sorted rows,
           their gradient, the weighted way back, and its gradient
  product  the experts' products on sorted rows: x W^T, with the gated
           activation, the gradients of rows and of weights
  adamw    one AdamW step over many tensors, states in 32 or in 8 bits

run() computes them in elementary torch operations in 32 bits, or, where the
module's `own` is set, through moe_expert_layer_ep_gb300.  exact() computes
the same from the definitions in 64 bits.
"""

import math

import torch

own = False

BLOCK = 128          # rows per expert are padded to this in the sorted layout
STATE_BLOCK = 256    # elements that share a scale of an 8-bit optimizer state
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # the smallest layer the repository runs: latency of plan and gather
        dict(name="sort_tiny", op="sort", way="sort", dtype="bf16", T=128, K=256, E=8, El=8, topk=2, skew=0.0, drop=0.0),
        # dispatch of the large prefill batch with popular experts
        dict(name="sort_large_skewed", op="sort", way="sort", dtype="bf16", T=8192, K=7168, E=256, El=256, topk=8,
             skew=1.2, drop=0.0),
        # the gradient of the dispatch on a rank that holds half of the experts, odd sizes, fp32 rows
        dict(name="sort_backward_odd", op="sort", way="sort_backward", dtype="fp32", T=1001, K=1001, E=40, El=20, topk=4,
             skew=0.5, drop=0.1),
        # one new token comes back from its experts
        dict(name="unsort_one_token", op="sort", way="unsort", dtype="bf16", T=1, K=7168, E=256, El=256, topk=8, skew=0.0,
             drop=0.0),
        # the combine's gradient, rows and weights, at the mid-size layer
        dict(name="unsort_backward", op="sort", way="unsort_backward", dtype="bf16", T=4096, K=2048, E=128, El=128, topk=8,
             skew=0.0, drop=0.05),
        # first product with the activation, mid-size layer, training batch
        dict(name="product_swiglu", op="product", way="swiglu", T=4096, C=2048, N=768, E=128, El=128, topk=8, skew=0.0),
        # second product of a few tokens on a rank with 32 of 256 experts: the weights' bytes count
        dict(name="product_few_rows", op="product", way="forward", T=16, C=2048, N=7168, E=256, El=32, topk=8, skew=0.0),
        # gradient through the second product and the activation, wide layer
        dict(name="product_dgrad_swiglu", op="product", way="dgrad_swiglu", T=2048, C=2048, N=7168, E=32, El=32, topk=8,
             skew=0.0),
        # gradient of the first product's weights, uneven experts
        dict(name="product_wgrad", op="product", way="wgrad", T=4096, C=2048, N=1536, E=128, El=128, topk=8, skew=0.3),
        # a small model's many small tensors: launches and latency count
        dict(name="adamw_small", op="adamw", param="fp32", grad="fp32", state=32, master=False, tensors=48, size=3000),
        # bf16 weights of the mid-size layer's experts, states in 32 bits
        dict(name="adamw_bf16", op="adamw", param="bf16", grad="bf16", state=32, master=False, tensors=16, size=9437184),
        # the same with a 32-bit copy of the weights and states in 8 bits
        dict(name="adamw_8bit", op="adamw", param="bf16", grad="bf16", state=8, master=True, tensors=16, size=18874368),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        most[c["op"]] = max(most.get(c["op"], 0.0), _cost(w))
    op = rng.choice(("sort", "product", "adamw"))
    while True:
        c = _drawn(rng, op)
        if _cost(work(c)) <= most[op]:
            return c


def _cost(w):
    return max(w["bytes"], w["flops"] / 50.0)


def _drawn(rng, op):
    if op == "adamw":
        param = rng.choice(("fp32", "bf16", "bf16"))
        tensors = _log_int(rng, 1, 300)
        return dict(op=op, param=param, grad=rng.choice((param, "bf16")), state=rng.choice((8, 32)),
                    master=param == "bf16" and rng.random() < 0.5, tensors=tensors,
                    size=_log_int(rng, 100, max(200, 300_000_000 // tensors)))
    E = rng.choice((4, 8, 16, 40, 64, 128, 256))
    El = E if rng.random() < 0.7 else max(1, E // rng.choice((2, 4, 8)))
    topk = rng.randint(1, min(8, E))
    if op == "sort":
        K = _log_int(rng, 16, 7168)
        return dict(op=op, way=rng.choice(("sort", "sort_backward", "unsort", "unsort_backward")),
                    dtype=rng.choice(("bf16", "bf16", "fp32")), T=_log_int(rng, 1, 8192),
                    K=K if rng.random() < 0.3 else -(-K // 8) * 8, E=E, El=El, topk=topk, skew=rng.choice((0.0, 0.5, 1.2)),
                    drop=rng.choice((0.0, 0.1)))
    while True:
        C, N = 8 * _log_int(rng, 8, 896), 8 * _log_int(rng, 8, 896)
        if 2 * El * C * N * 2 <= 2_000_000_000:
            break
    return dict(op=op, way=rng.choice(("forward", "swiglu", "dgrad", "dgrad_swiglu", "wgrad")), T=_log_int(rng, 1, 8192),
                C=C, N=N, E=E, El=El, topk=topk, skew=rng.choice((0.0, 0.3)))


# --------------------------------------------------------------------------- inputs
def _routing(T, E, topk, skew, g):
    """Each token's topk experts, more often the popular ones (popularity r^-skew of rank r), and softmax weights."""
    z = torch.randn((T, E), generator=g, device="cuda")
    rank = torch.randperm(E, generator=g, device="cuda").float() + 1.0
    v, ids = torch.topk(z - skew * torch.log(rank), topk, dim=1)
    return ids.to(torch.int32), torch.softmax(v, 1)


def _plan(ids, El):
    """The sorted layout of the routing: destination row of each assignment (-1: dropped or not local), each expert's
    first row and its number of rows."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < El), flat, El)
    order = torch.sort(key, stable=True).indices
    counts = torch.zeros(El + 1, dtype=torch.long, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    padded = (counts + BLOCK - 1) // BLOCK * BLOCK
    start = torch.cumsum(padded, 0) - padded
    first = torch.cumsum(counts, 0) - counts
    sorted_key = key[order]
    dst = start[sorted_key] + torch.arange(flat.numel(), device=ids.device) - first[sorted_key]
    dst = torch.where(sorted_key < El, dst, -1)
    src2dst = torch.empty_like(flat).scatter_(0, order, dst)
    return src2dst.to(torch.int32).view(ids.shape), start[:El].to(torch.int32), counts[:El].to(torch.int32)


def _rows_bound(A, El):
    nonempty = min(A, El)
    return BLOCK * (nonempty + (A - nonempty) // BLOCK)


def _sizes(case):
    """The adamw tensors' sizes: ragged around case["size"], from the case alone."""
    n = case["tensors"]
    return [max(1, int(case["size"] * (0.25 + 1.5 * i / max(1, n - 1))) - 7 * (i % 3)) for i in range(n)]


def _places(case):
    """Where each adamw tensor begins in the program's buffers (each kind of value in one buffer, every tensor at a
    whole block), and the buffers' length."""
    at, sizes = [0], _sizes(case)
    for n in sizes:
        at.append(at[-1] + -(-n // STATE_BLOCK) * STATE_BLOCK)
    return at[:-1], sizes, at[-1]


def _views(buf, case):
    at, sizes, _ = _places(case)
    return [buf[a : a + n] for a, n in zip(at, sizes)]


def _adamw_inputs(case, g):
    at, sizes, total = _places(case)
    real = torch.zeros(total, dtype=torch.bool, device="cuda")
    for a, n in zip(at, sizes):
        real[a : a + n] = True

    def randn(scale):
        return torch.randn(total, generator=g, device="cuda").mul_(scale).masked_fill_(~real, 0.0)

    flat = {"p": randn(0.02)}
    flat["g"] = randn(1e-3).to(DTYPES[case["grad"]])
    flat["m"], flat["v"] = randn(3e-4), randn(1e-3).square_()
    if case["master"]:
        flat["p32"] = flat["p"].clone()
    flat["p"] = flat["p"].to(DTYPES[case["param"]])
    if case["state"] == 8:
        flat["m"], flat["ms"] = _encode_m(flat["m"])
        flat["v"], flat["vs"] = _encode_v(flat["v"])
    s = {"flat": flat}
    for k in ("p", "p32", "g", "m", "v"):
        if k in flat:
            s[k] = _views(flat[k], case)
    for k in ("ms", "vs"):
        if k in flat:
            s[k] = [flat[k][a // STATE_BLOCK : a // STATE_BLOCK + -(-n // STATE_BLOCK)] for a, n in zip(at, sizes)]
    return s


def _prepare_sort(case, s, g):
    T, K, El, dt = case["T"], case["K"], case["El"], DTYPES[case["dtype"]]
    s["ids"], s["w"] = _routing(T, case["E"], case["topk"], case["skew"], g)
    if case["drop"]:
        s["ids"].masked_fill_(torch.rand(s["ids"].shape, generator=g, device="cuda") < case["drop"], -1)
    s["rows"] = _rows_bound(T * case["topk"], El)
    s["src2dst"], _, _ = _plan(s["ids"], El)
    # sorted rows; padding rows are never written, and stay zero.  The last row takes what is dropped in the plain form.
    s["sorted"] = torch.zeros((s["rows"] + 1, K), dtype=dt, device="cuda")
    if case["way"] in ("sort", "unsort_backward"):
        s["x"] = torch.randn((T, K), generator=g, device="cuda").to(dt)
    if case["way"] != "sort":
        s["y"] = torch.randn((s["rows"], K), generator=g, device="cuda").to(dt)


def _prepare_product(case, s, g):
    C, N, El, way = case["C"], case["N"], case["El"], case["way"]
    ids, _ = _routing(case["T"], case["E"], case["topk"], case["skew"], g)
    _, s["start"], s["counts"] = _plan(ids, El)
    rows = _rows_bound(ids.numel(), El)
    # rows that carry a token, and their places among El equally tall experts
    counts, start = s["counts"].tolist(), s["start"].tolist()
    s["tall"] = max(max(counts), 1)
    at = [torch.arange(n, device="cuda") for n in counts]
    s["valid"] = torch.cat([a + b for a, b in zip(at, start)])
    s["place"] = torch.cat([a + e * s["tall"] for e, a in enumerate(at)])
    s["status"] = torch.zeros(4, dtype=torch.int32, device="cuda")

    def rand(r, c):
        return torch.randn((r, c), generator=g, device="cuda").to(torch.bfloat16)

    def zeros(r, c):
        return torch.zeros((r, c), dtype=torch.bfloat16, device="cuda")   # padding rows stay as they are

    wide = 2 * N if way == "swiglu" else N
    if way != "wgrad":
        s["w"] = torch.empty((El, wide, C), dtype=torch.bfloat16, device="cuda").normal_(0.0, 0.02, generator=g)
    if way in ("forward", "swiglu", "wgrad"):
        s["x"] = rand(rows, C)
    if way in ("dgrad", "dgrad_swiglu", "wgrad"):
        s["dy"] = rand(rows, N)
    if way == "dgrad_swiglu":
        s["gu"] = rand(rows, 2 * C)
        s["out"] = zeros(rows, 2 * C)
    elif way == "dgrad":
        s["out"] = zeros(rows, C)
    elif way == "swiglu":
        s["out"], s["h"] = zeros(rows, 2 * N), zeros(rows, N)
    elif way == "forward":
        s["out"] = zeros(rows, N)
    else:
        s["out"] = torch.zeros((El, N, C), dtype=torch.bfloat16, device="cuda")


HYPER = dict(step=10, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "sort":
        _prepare_sort(case, s, g)
    elif case["op"] == "product":
        _prepare_product(case, s, g)
    else:
        s.update(_adamw_inputs(case, g))
        s["grad_scale"] = torch.rand(1, generator=g, device="cuda") * 0.5 + 0.5   # what gradient clipping gives
        if own:   # the optimizer's handle: the tensors' places, as a program keeps them
            import moe_expert_layer_ep_gb300 as M
            s["opt"] = M.moe_adamw_create(s["p"], s["g"], s["m"], s["v"], masters=s.get("p32"), avg_scales=s.get("ms"),
                                          sq_scales=s.get("vs"))
    return s


# --------------------------------------------------------------------------- the plain forms
def _gathered(s, src2dst):
    """y's rows of each assignment in 32 bits, zeros for dropped ones: [T, topk, K]."""
    kept = (src2dst >= 0).unsqueeze(-1)
    y = s["y"][src2dst.clamp(min=0).long()].float()
    return torch.where(kept, y, torch.zeros_like(y))


def _put(s, src2dst, values):
    """values [T, topk, K] to the sorted rows (dropped ones to the spare last row)."""
    at = torch.where(src2dst >= 0, src2dst, s["rows"]).long().reshape(-1)
    s["sorted"].index_copy_(0, at, values.reshape(at.numel(), -1))
    return s["sorted"][: s["rows"]]


def _plain_sort(s, way):
    if way == "sort":
        src2dst, start, counts = _plan(s["ids"], s["case"]["El"])
        x = s["x"].unsqueeze(1).expand(-1, src2dst.shape[1], -1)
        return {"sorted": _put(s, src2dst, x), "src2dst": src2dst, "start": start, "counts": counts}
    y = _gathered(s, s["src2dst"])
    if way == "sort_backward":
        return {"dx": y.sum(1).to(s["y"].dtype)}
    if way == "unsort":
        return {"out": (y * s["w"].unsqueeze(-1)).sum(1).to(s["y"].dtype)}
    d = s["x"].float().unsqueeze(1)
    dy = (d * s["w"].unsqueeze(-1)).to(s["y"].dtype)
    return {"dy": _put(s, s["src2dst"], dy), "dw": (d * y).sum(-1)}


def _spread(s, x):
    """Rows that carry a token in 32 bits, as [experts, tallest expert's rows, columns]."""
    El = s["case"]["El"]
    out = torch.zeros((El * s["tall"], x.shape[1]), dtype=torch.float32, device=x.device)
    out[s["place"]] = x[s["valid"]].float()
    return out.view(El, s["tall"], -1)


def _back(s, y, out):
    """[experts, rows, columns] to the sorted rows of out, rounded once."""
    out[s["valid"]] = y.reshape(-1, y.shape[-1])[s["place"]].to(out.dtype)
    return out


def _plain_product(s, way):
    if way == "wgrad":
        dw = torch.bmm(_spread(s, s["dy"]).transpose(1, 2), _spread(s, s["x"]))
        return {"dw": dw.to(torch.bfloat16)}
    w = s["w"].float()
    if way in ("forward", "swiglu"):
        y = torch.bmm(_spread(s, s["x"]), w.transpose(1, 2))
        if way == "forward":
            return {"y": _back(s, y, s["out"])}
        gate, up = y.chunk(2, dim=-1)
        return {"gu": _back(s, y, s["out"]), "h": _back(s, gate / (1.0 + torch.exp(-gate)) * up, s["h"])}
    d = torch.bmm(_spread(s, s["dy"]), w)
    if way == "dgrad":
        return {"dx": _back(s, d, s["out"])}
    gate, up = _spread(s, s["gu"]).chunk(2, dim=-1)
    sig = 1.0 / (1.0 + torch.exp(-gate))
    dg = d * up * sig * (1.0 + gate * (1.0 - sig))
    return {"dgu": _back(s, torch.cat((dg, d * gate * sig), -1), s["out"])}


def _scales(t):
    """The largest |t| of each block (at least the smallest normal number, where it is not zero), and its reciprocal."""
    s = t.view(-1, STATE_BLOCK).abs().amax(1)
    s = torch.where(s > 0, s.clamp(min=2.0**-126), s)
    return s, torch.where(s > 0, 1.0 / s, 0.0)


def _encode_m(t):
    s, inv = _scales(t)
    share = (t.abs().view(-1, STATE_BLOCK) * inv.unsqueeze(1)).view(-1)
    c = torch.round(torch.sqrt(share) * 127.0)
    return torch.where(t < 0, -c, c).to(torch.int8), s


def _encode_v(t):
    s, inv = _scales(t)
    root = (torch.sqrt(t).view(-1, STATE_BLOCK) * torch.sqrt(inv).unsqueeze(1)).view(-1)
    c = torch.round(torch.sqrt(root) * 255.0)
    return torch.where(t > 0, c.clamp(min=1.0), c).to(torch.uint8), s


def _decode_m(c, s):
    r = c.to(s.dtype) * (1.0 / 127.0)
    return ((r * r.abs()).view(-1, STATE_BLOCK) * s.unsqueeze(1)).view(-1)


def _decode_v(c, s):
    r = c.to(s.dtype) * (1.0 / 255.0)
    r = r * r
    return ((r * r).view(-1, STATE_BLOCK) * s.unsqueeze(1)).view(-1)


def _plain_adamw(f, grad_scale):
    """On the program's whole buffers: the gaps between tensors are zeros and stay zeros."""
    h, coded = HYPER, "ms" in f
    p = f["p32"] if "p32" in f else f["p"].float()
    g = f["g"].float() * grad_scale
    m = (_decode_m(f["m"], f["ms"]) if coded else f["m"]) * h["beta1"] + g * (1.0 - h["beta1"])
    v = (_decode_v(f["v"], f["vs"]) if coded else f["v"]) * h["beta2"] + g * g * (1.0 - h["beta2"])
    denom = torch.sqrt(v) * (1.0 / math.sqrt(1.0 - h["beta2"] ** h["step"])) + h["eps"]
    p = p * (1.0 - h["lr"] * h["weight_decay"]) - m / denom * (h["lr"] / (1.0 - h["beta1"] ** h["step"]))
    f["p"].copy_(p)
    if "p32" in f:
        f["p32"].copy_(p)
    if not coded:
        f["m"].copy_(m)
        f["v"].copy_(v)
        return
    for k, (c, x) in (("m", _encode_m(m)), ("v", _encode_v(v))):
        f[k].copy_(c)
        f[k + "s"].copy_(x)


# --------------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if case["op"] == "adamw":
        if own:
            import moe_expert_layer_ep_gb300 as M
            M.moe_adamw_step(s["opt"], grad_scale=s["grad_scale"], **HYPER)
        else:
            _plain_adamw(s["flat"], s["grad_scale"])
        return _adamw_outputs(s["flat"])
    if not own:
        return _plain_sort(s, case["way"]) if case["op"] == "sort" else _plain_product(s, case["way"])
    import moe_expert_layer_ep_gb300 as M
    way = case["way"]
    if case["op"] == "sort":
        if way == "sort":
            src2dst, start, counts = M.moe_sort_plan(s["ids"], case["E"], case["El"])
            out = M.moe_sort_tokens(s["x"], src2dst, out=s["sorted"][: s["rows"]])
            return {"sorted": out, "src2dst": src2dst, "start": start, "counts": counts}
        if way == "sort_backward":
            return {"dx": M.moe_unsort_tokens(s["y"], s["src2dst"])}
        if way == "unsort":
            return {"out": M.moe_unsort_tokens(s["y"], s["src2dst"], s["w"])}
        dy, dw = M.moe_unsort_tokens_backward(s["x"], s["y"], s["src2dst"], s["w"], dy=s["sorted"][: s["rows"]])
        return {"dy": dy, "dw": dw}
    at = (s["start"], s["counts"], s["status"])
    if way == "forward":
        return {"y": M.moe_expert_gemm(s["x"], s["w"], *at, y=s["out"])}
    if way == "swiglu":
        h, gu = M.moe_expert_gemm_swiglu(s["x"], s["w"], *at, h=s["h"], gu=s["out"])
        return {"gu": gu, "h": h}
    if way == "dgrad":
        return {"dx": M.moe_expert_gemm_dgrad(s["dy"], s["w"], *at, dx=s["out"])}
    if way == "dgrad_swiglu":
        return {"dgu": M.moe_expert_gemm_dgrad_swiglu(s["dy"], s["w"], s["gu"], *at, dgu=s["out"])}
    return {"dw": M.moe_expert_gemm_wgrad(s["dy"], s["x"], *at, dw=s["out"])}


def _adamw_outputs(f):
    """The updated buffers, whole.  A state in 8 bits stands for the signed root of its value's share of the block's
    scale (the fourth root for v); those numbers, -127..127 and 0..255, are given exactly in bfloat16."""
    out = {k: f[k] for k in ("p", "p32", "m", "v", "ms", "vs") if k in f}
    if "ms" in f:
        out["m"], out["v"] = f["m"].to(torch.bfloat16), f["v"].to(torch.bfloat16)
    return out


# --------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    w = work(case)
    if w["flops"] > 4e12 or w["bytes"] > 4e10:
        return None
    s = prepare(case, seed)
    if case["op"] == "sort":
        return _exact_sort(s, case)
    return _exact_product(s, case) if case["op"] == "product" else _exact_adamw(s)


def _exact_sort(s, case):
    way, T, K = case["way"], case["T"], case["K"]
    dst = s["src2dst"].long()
    if way == "sort":
        out = torch.zeros((s["rows"], K), dtype=torch.float64, device="cuda")
        for j in range(case["topk"]):
            kept = dst[:, j] >= 0
            out[dst[kept, j]] = s["x"][kept].double()
        return {"sorted": out, "src2dst": None, "start": None, "counts": None}
    y = s["y"].double()
    if way in ("sort_backward", "unsort"):
        out = torch.zeros((T, K), dtype=torch.float64, device="cuda")
        for j in range(case["topk"]):
            kept = dst[:, j] >= 0
            rows = y[dst[kept, j]]
            out[kept] += rows if way == "sort_backward" else rows * s["w"][kept, j].double().unsqueeze(1)
        return {"dx" if way == "sort_backward" else "out": out}
    d = s["x"].double()
    dy, dw = torch.zeros_like(y), torch.zeros((T, case["topk"]), dtype=torch.float64, device="cuda")
    for j in range(case["topk"]):
        kept = dst[:, j] >= 0
        dy[dst[kept, j]] = d[kept] * s["w"][kept, j].double().unsqueeze(1)
        dw[kept, j] = torch.einsum("tk,tk->t", d[kept], y[dst[kept, j]])
    return {"dy": dy, "dw": dw}


def _exact_product(s, case):
    way, out = case["way"], {}
    if way == "wgrad":
        dw = torch.zeros((case["El"], case["N"], case["C"]), dtype=torch.float64, device="cuda")
    for e, (a, n) in enumerate(zip(s["start"].tolist(), s["counts"].tolist())):
        if n == 0:
            continue
        r = slice(a, a + n)
        if way == "wgrad":
            dw[e] = s["dy"][r].double().T @ s["x"][r].double()
            continue
        w = s["w"][e].double()
        if way == "forward":
            got = {"y": s["x"][r].double() @ w.T}
        elif way == "swiglu":
            gate, up = s["x"][r].double() @ w[: case["N"]].T, s["x"][r].double() @ w[case["N"] :].T
            got = {"gu": torch.cat((gate, up), 1), "h": gate * torch.sigmoid(gate) * up}
        else:
            d = s["dy"][r].double() @ w
            got = {"dx": d}
            if way == "dgrad_swiglu":
                gate, up = s["gu"][r].double().split(case["C"], 1)
                sig = torch.sigmoid(gate)
                got = {"dgu": torch.cat((d * up * (sig + gate * sig * (1 - sig)), d * gate * sig), 1)}
        for k, v in got.items():
            if k not in out:
                rows = (s["x"] if "x" in s else s["dy"]).shape[0]
                out[k] = torch.zeros((rows, v.shape[1]), dtype=torch.float64, device="cuda")
            out[k][r] = v
    if way == "wgrad":
        return {"dw": dw}
    return {k: out[k] for k in {"forward": ("y",), "swiglu": ("gu", "h"), "dgrad": ("dx",), "dgrad_swiglu": ("dgu",)}[way]
            if k in out}


def _exact_adamw(s):
    f, h = s["flat"], HYPER
    coded = "ms" in f

    def state(k, power):
        if not coded:
            return f[k].double()
        root = f[k].double() / (127.0 if k == "m" else 255.0)
        return torch.sign(root) * root.abs() ** power * f[k + "s"].double().repeat_interleave(STATE_BLOCK)

    g = f["g"].double() * s["grad_scale"].double()
    m = state("m", 2).mul_(h["beta1"]).add_(g, alpha=1 - h["beta1"])
    v = state("v", 4).mul_(h["beta2"]).addcmul_(g, g, value=1 - h["beta2"])
    p = f["p32" if "p32" in f else "p"].double() * (1 - h["lr"] * h["weight_decay"])
    mhat, vhat = m / (1 - h["beta1"] ** h["step"]), v / (1 - h["beta2"] ** h["step"])
    p.sub_(mhat.div_(vhat.sqrt_().add_(h["eps"])), alpha=h["lr"])
    out = {"p": p}
    if "p32" in f:
        out["p32"] = p
    if not coded:
        return {**out, "m": m, "v": v}
    for k, x, levels, root in (("m", m, 127.0, 0.5), ("v", v, 255.0, 0.25)):
        top = x.view(-1, STATE_BLOCK).abs().amax(1)
        share = x.abs() / top.clamp(min=1e-300).repeat_interleave(STATE_BLOCK)
        c = torch.round(share.pow_(root).mul_(levels))
        out[k] = torch.sign(x) * (c.clamp_(min=1.0) if k == "v" else c)
        out[k + "s"] = top
    return {k: out[k] for k in ("p", "p32", "m", "v", "ms", "vs") if k in out}


# --------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    """Bytes: each input read once, each output written once; operations of the products and sums.  Rows that stay on
    this rank are counted by their share El / E; an expert's weights where some token is expected to choose it."""
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        size = {"fp32": 4, "bf16": 2}
        per = size[case["grad"]] + (size[case["param"]] + 8 if case["master"] else 2 * size[case["param"]])
        per += 16 if case["state"] == 32 else 4 + 16 / STATE_BLOCK
        return {"bytes": n * per, "flops": n * 15}
    T, E, El, topk = case["T"], case["E"], case["El"], case["topk"]
    kept = T * topk * El / E
    if case["op"] == "sort":
        es, K, way = 4 if case["dtype"] == "fp32" else 2, case["K"], case["way"]
        kept *= 1.0 - case["drop"]
        rows = {"sort": T + kept, "sort_backward": T + kept, "unsort": T + kept, "unsort_backward": T + 2 * kept}[way]
        small = {"sort": 8, "sort_backward": 4, "unsort": 8, "unsort_backward": 12}[way] * T * topk
        ops = {"sort": 0, "sort_backward": 1, "unsort": 2, "unsort_backward": 3}[way]
        return {"bytes": rows * K * es + small, "flops": kept * K * ops}
    C, N, way = case["C"], case["N"], case["way"]
    wide = 2 * N if way == "swiglu" else N
    weights = El * (1.0 - (1.0 - topk / E) ** T) * wide * C * 2
    if way == "wgrad":
        weights = El * N * C * 2
    # columns of sorted rows in and out
    cols = {"forward": C + N, "swiglu": C + 3 * N, "dgrad": N + C, "dgrad_swiglu": N + 4 * C, "wgrad": N + C}[way]
    return {"bytes": weights + kept * cols * 2, "flops": 2.0 * kept * wide * C}
