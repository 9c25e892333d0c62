"""The token-score operators from their definitions in 64 bits, one row at a
time, on the CPU: what the kernels' outputs are held against.  Scores come as
float64 numpy rows (the exact values of fp32 or bf16 scores)."""
import numpy as np

INF = float("inf")


def bad(x):
    """A NaN or +inf among the scores."""
    return bool(np.isnan(x).any() or (x == INF).any())


def lse_parts(y):
    """(max, log sum exp relative to it); (-inf, 0) for nothing but -inf."""
    if bad(y):
        return np.nan, np.nan
    m = y.max()
    if m == -INF:
        return -INF, 0.0
    return m, float(np.log(np.exp(y - m).sum()))


def log_softmax(y):
    m, s = lse_parts(y)
    if m != m:
        return np.full_like(y, np.nan)
    if m == -INF:
        return np.full_like(y, -INF)
    return (y - m) - s


def logprob_row(x, token, scale, k):
    """(logprob, entropy, stats, top_ids, top_logprob) of one row."""
    if token is not None and token < 0:
        return 0.0, 0.0, (-INF, 0.0), [-1] * k, [-INF] * k
    y = x * scale
    lp = log_softmax(y)
    if bad(x):
        h = np.nan
    else:
        live = lp > -INF
        h = float(-(np.exp(lp[live]) * lp[live]).sum())
    got = np.nan if token is None or token >= x.size else lp[token]
    key = np.where(np.isnan(x), INF, x)
    order = sorted(range(x.size), key=lambda i: (not np.isnan(x[i]), -key[i], i))[:k] if k else []
    return got, h, lse_parts(y), order, [lp[i] for i in order]


def logprob_grad_row(x, token, scale, g_lp, g_h):
    n = x.size
    if token is not None and token < 0:
        return np.zeros(n)
    if bad(x) or (token is not None and token >= n):
        return np.full(n, np.nan)
    lp = log_softmax(x * scale)
    p = np.exp(lp)
    live = lp > -INF
    h = -(p[live] * lp[live]).sum()
    one = np.zeros(n)
    if token is not None:
        one[token] = 1.0
    out = np.zeros(n)
    out[live] = scale * (g_lp * (one[live] - p[live]) - g_h * p[live] * (lp[live] + h))
    return out


def teacher(val, tail, t_scale):
    """log q, q, remaining mass; None where the row has nothing to learn from."""
    if tail:
        q = np.exp(val)
        return val, q, np.nan if np.isnan(q.sum()) else max(0.0, 1.0 - q.sum())
    v = val * t_scale
    if np.isnan(v).any():
        return np.full_like(v, np.nan), np.full_like(v, np.nan), 0.0
    if v.max() == -INF:
        return None
    logq = log_softmax(v)
    return logq, np.exp(logq), 0.0


def distill_row(x, ids, val, scale, tail, t_scale, g):
    """(loss, stats, gradient, magnitude of the loss's terms) of one row."""
    n = x.size
    keep = ids >= 0
    if not keep.any():
        return 0.0, (-INF, 0.0, -INF, 0.0), np.zeros(n), 0.0
    ids, val = ids[keep], np.where(ids[keep] >= n, np.nan, val[keep])
    here = ids[ids < n]
    y = x * scale
    rest = y.copy()
    rest[here] = -INF
    stats = lse_parts(y) + lse_parts(rest)
    t = teacher(val, tail, t_scale)
    if t is None:
        return 0.0, stats, np.zeros(n), 0.0
    logq, q, q_rest = t
    if bad(x) or np.isnan(val).any():
        return np.nan, stats, np.full(n, np.nan), 1.0
    lp = log_softmax(y)
    on = q > 0
    with np.errstate(invalid="ignore"):
        terms = q[on] * (logq[on] - lp[ids][on])
    loss, size = terms.sum(), (q[on] * (np.abs(logq[on]) + np.abs(lp[ids][on]) + 1)).sum()
    log_p_rest = -INF if stats[2] == -INF else (stats[2] - stats[0]) + (stats[3] - stats[1])
    if q_rest > 0:
        loss += q_rest * (np.log(q_rest) - log_p_rest)
        size += q_rest * (abs(np.log(q_rest)) + abs(log_p_rest) + 1)
    p = np.exp(lp)
    grad = p * (q.sum() + q_rest)
    grad[ids] -= q
    if stats[2] > -INF:
        grad -= np.exp((rest - stats[2]) - stats[3]) * q_rest     # in this order: m may be the type's lowest value
    grad[x == -INF] = 0.0
    return float(loss), stats, grad * scale * g, size
