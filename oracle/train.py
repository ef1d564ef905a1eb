"""Training of the experts in fp64: tokens sorted by expert and back, the
experts' products with their activations, biases and residuals, the router's
losses, one AdamW step, and the gradients.  Plain loops over assignments and experts; inputs are the values the
CUDA path gets, outputs are not rounded to its storage types.
"""

import math

import numpy as np

STATE_BLOCK = 256


# ---------------------------------------------------------------- rows
def sort_plan(ids, E_global, E_local, expert_start):
    """(src2dst [T, k], start [E_local], counts [E_local]): assignments in
    t * k + j order per expert, experts from multiples of 128 rows."""
    ids = np.asarray(ids)
    flat = ids.reshape(-1)
    local = np.where((flat >= 0) & (flat < E_global), flat - expert_start, -1)
    local = np.where((local >= 0) & (local < E_local), local, -1)
    counts = np.zeros(E_local, dtype=np.int64)
    rank = np.full(flat.size, -1, dtype=np.int64)
    for i, e in enumerate(local):
        if e >= 0:
            rank[i] = counts[e]
            counts[e] += 1
    start = np.zeros(E_local, dtype=np.int64)
    for e in range(1, E_local):
        start[e] = start[e - 1] + -(-counts[e - 1] // 128) * 128
    dst = np.array([start[e] + r if e >= 0 else -1 for e, r in zip(local, rank)], dtype=np.int64)
    return dst.reshape(ids.shape), start, counts


def sort_tokens(x, src2dst, sorted_rows):
    """sorted_rows with x's rows put in their places."""
    out = np.array(sorted_rows, dtype=np.float64)
    for (t, j), d in np.ndenumerate(src2dst):
        if 0 <= d < len(out):
            out[d] = x[t]
    return out


def unsort_tokens(y, src2dst, w=None):
    out = np.zeros((src2dst.shape[0], y.shape[1]))
    for (t, j), d in np.ndenumerate(src2dst):
        if 0 <= d < len(y):
            out[t] += (1.0 if w is None else float(w[t, j])) * y[d]
    return out


def unsort_tokens_backward(dout, y, src2dst, w, sorted_rows):
    dy, dw = np.array(sorted_rows, dtype=np.float64), np.zeros(src2dst.shape)
    for (t, j), d in np.ndenumerate(src2dst):
        if 0 <= d < len(y):
            dy[d] = float(w[t, j]) * dout[t]
            dw[t, j] = float(np.dot(dout[t], y[d]))
    return dy, dw


# ---------------------------------------------------------------- products
def _segments(start, counts):
    return [(e, slice(int(a), int(a) + int(n))) for e, (a, n) in enumerate(zip(start, counts)) if n > 0]


def expert_gemm(x, w, start, counts):
    """y[r] = x[r] w_e^T for the rows of each expert; NaN elsewhere."""
    y = np.full((x.shape[0], w.shape[1]), np.nan)
    for e, r in _segments(start, counts):
        y[r] = x[r] @ w[e].T
    return y


def expert_gemm_dgrad(dy, w, start, counts):
    dx = np.full((dy.shape[0], w.shape[2]), np.nan)
    for e, r in _segments(start, counts):
        dx[r] = dy[r] @ w[e]
    return dx


def expert_gemm_wgrad(dy, x, start, counts):
    dw = np.zeros((len(counts), dy.shape[1], x.shape[1]))
    for e, r in _segments(start, counts):
        dw[e] = dy[r].T @ x[r]
    return dw


def swiglu(gu):
    g, u = np.split(gu, 2, axis=1)
    return g / (1.0 + np.exp(-g)) * u


def swiglu_backward(dh, gu):
    g, u = np.split(gu, 2, axis=1)
    s = 1.0 / (1.0 + np.exp(-g))
    return np.concatenate([dh * u * s * (1.0 + g * (1.0 - s)), dh * g * s], axis=1)


_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def _sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def act(name, z):
    """(value, derivative) of an activation."""
    z = np.asarray(z, dtype=np.float64)
    if name == "none":
        return z, np.ones_like(z)
    if name == "silu":
        s = _sigmoid(z)
        return z * s, s * (1.0 + z * (1.0 - s))
    if name == "gelu":
        cdf = 0.5 * _erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        c = 2.0 * math.sqrt(2.0 / math.pi)
        s = _sigmoid(c * (z + 0.044715 * z ** 3))
        return z * s, s + z * s * _sigmoid(-c * (z + 0.044715 * z ** 3)) * c * (1.0 + 3 * 0.044715 * z * z)
    r = np.maximum(z, 0.0)
    return (r, (z > 0).astype(np.float64)) if name == "relu" else (r * r, 2.0 * r)


def expert_bias_grad(dy, start, counts):
    db = np.zeros((len(counts), dy.shape[1]))
    for e, r in _segments(start, counts):
        db[e] = dy[r].sum(axis=0)
    return db


# ---------------------------------------------------------------- router
def route_losses(logits, ids, kept=None):
    """(balance, size): E sum_e f_e P_e, f_e the share of the assignments that went to e (those that were kept) and P_e
    the mean probability of e, and the mean square of the logits' logsumexp; means over the tokens that have an id."""
    ids = np.asarray(ids)
    kept = ids >= 0 if kept is None else (ids >= 0) & np.asarray(kept, dtype=bool)
    T, E = logits.shape
    there = (ids >= 0).any(axis=1)
    n = max(1, int(there.sum()))
    f = np.zeros(E)
    for e in ids[kept]:
        f[e] += 1.0 / (n * ids.shape[1])
    top = logits.max(axis=1, keepdims=True)
    lse = top[:, 0] + np.log(np.exp(logits - top).sum(axis=1))
    p = np.exp(logits - lse[:, None])
    return E * float((f * p[there].sum(axis=0)).sum()) / n, float((lse[there] ** 2).sum()) / n


def route_backward(logits, ids, weights, dweights, balance, zloss, kept=None):
    """Gradient to the logits of balance * the first loss + zloss * the second + sum(dweights * weights), weights the
    softmax over a token's ids that are not -1; with kept, the sum runs over the kept assignments alone."""
    ids = np.asarray(ids)
    kept = ids >= 0 if kept is None else (ids >= 0) & np.asarray(kept, dtype=bool)
    T, E = logits.shape
    k = ids.shape[1]
    there = (ids >= 0).any(axis=1)
    n = max(1, int(there.sum()))
    f = np.zeros(E)
    for e in ids[kept]:
        f[e] += 1.0 / (n * k)
    dz = np.zeros((T, E))
    for t in range(T):
        if not there[t]:
            continue
        z = logits[t]
        lse = z.max() + math.log(np.exp(z - z.max()).sum())
        p = np.exp(z - lse)
        dz[t] = balance * E / n * p * (f - (f * p).sum()) + zloss * 2.0 * lse / n * p
        mean = sum(weights[t, j] * dweights[t, j] for j in range(k) if kept[t, j])
        for j in range(k):
            if ids[t, j] >= 0:
                dz[t, ids[t, j]] += weights[t, j] * ((dweights[t, j] if kept[t, j] else 0.0) - mean)
    return dz


# ---------------------------------------------------------------- optimizer
def adamw(p, g, m, v, step, lr, beta1, beta2, eps, weight_decay, grad_scale=1.0):
    """(p, m, v) after one step."""
    g = g * grad_scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    mhat, vhat = m / (1 - beta1 ** step), v / (1 - beta2 ** step)
    return p * (1 - lr * weight_decay) - lr * mhat / (np.sqrt(vhat) + eps), m, v


def _per_block(x):
    n = x.size
    pad = np.zeros(-(-n // STATE_BLOCK) * STATE_BLOCK)
    pad[:n] = np.abs(x)
    return pad.reshape(-1, STATE_BLOCK).max(axis=1)


def state_scales(x):
    """Largest magnitude of each 256 consecutive elements, at least 2^-126 where not 0."""
    s = _per_block(x)
    return np.where(s > 0, np.maximum(s, 2.0 ** -126), s)


def state_roots(x, power, levels, scales):
    """The unrounded codes: levels * sign(x) * (|x| / s)^(1/power)."""
    s = np.repeat(scales, STATE_BLOCK)[: x.size]
    share = np.divide(np.abs(x), s, out=np.zeros_like(x), where=s > 0)
    return np.sign(x) * levels * share ** (1.0 / power)


def state_values(codes, power, levels, scales):
    s = np.repeat(np.asarray(scales, dtype=np.float64), STATE_BLOCK)[: codes.size]
    r = np.asarray(codes, dtype=np.float64) / levels
    return np.sign(r) * np.abs(r) ** power * s
