"""Training of the experts in fp64: tokens sorted by expert and back, the
experts' products with their gated activation, one AdamW step, and the
gradients.  Plain loops over assignments and experts; inputs are the values the
CUDA path gets, outputs are not rounded to its storage types.
"""

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
