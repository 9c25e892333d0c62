"""The embedding's gradient, the adjusted scores and the gradient norm from
their definitions in 64 bits, on the CPU: what the kernels' outputs are held
against.  Values come as float64 numpy arrays (the exact values of fp32 or bf16
ones); bounds are what the definition's own fp32 steps may be off."""
import numpy as np

INF = float("inf")
U = 2.0 ** -24                  # half an fp32 step
HALF_STEP = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8}
LEAST = {"fp32": 2.0 ** -149, "bf16": 2.0 ** -133}      # the smallest step, below the normal range


def rounded(want, dtype):
    """How far the rounding of `want` to dtype may be off."""
    w = np.where(np.isfinite(want), np.abs(want), 0.0)
    return w * HALF_STEP[dtype] + LEAST[dtype]


def in_type(want, dtype):
    """What lies beyond the type's largest value by half a step or more rounds to an infinity."""
    most = 2.0 ** 127 * (2 - HALF_STEP[dtype])
    with np.errstate(invalid="ignore"):
        return np.where(np.abs(want) >= most, np.copysign(INF, want), want)


def embedding_grad(g, ids, vocab, scale, old):
    """(gradient, bound before the rounding to the type).  An fp32 sum of n
    terms is off by at most n U sum |g| in any order, the product by U, the
    addition to what was there by U of its result."""
    want = np.zeros((vocab, g.shape[1]))
    size, n = np.zeros_like(want), np.zeros(vocab)
    on = (ids >= 0) & (ids < vocab)
    np.add.at(want, ids[on], g[on])
    np.add.at(size, ids[on], np.abs(g[on]))
    np.add.at(n, ids[on], 1)
    s = abs(scale)
    bound = (n[:, None] + 2) * U * size * s * 1.01
    want *= scale
    if old is not None:
        bound = bound + U * np.abs(want + old) * 1.01
        want = want + old
    bound[np.arange(vocab)[n == 0]] = 0.0
    return want, bound, n == 0


def adjusted_row(x, history, n_prompt, rep, freq, pres, bias_ids, bias, allowed):
    """(scores, bound before the rounding): each step is off by U of its result."""
    V = x.size
    y = x.copy()
    bound = np.zeros(V)
    history = np.asarray(history, dtype=np.int64)
    there = (history >= 0) & (history < V)
    said = there & (np.arange(history.size) >= n_prompt)
    seen = np.unique(history[there])
    times = np.bincount(history[said], minlength=V)
    with np.errstate(all="ignore"):
        if rep is not None:
            up = x[seen] > 0
            y[seen] = np.where(up, x[seen] / rep, x[seen] * rep)
            bound[seen] += U * np.abs(y[seen])
        c = np.nonzero(times)[0]
        if freq is not None:
            y[c] -= freq * times[c]
            bound[c] += U * (np.abs(freq * times[c]) + np.abs(y[c]))
        if pres is not None:
            y[c] -= pres
            bound[c] += U * np.abs(y[c])
        sums, sizes = {}, {}
        for i, b in zip(bias_ids, bias):
            if 0 <= i < V:
                sums[i] = sums.get(i, 0.0) + b
                sizes[i] = sizes.get(i, 0.0) + abs(b)
                bound[i] += U * sizes[i]
        for i, b in sums.items():
            y[i] += b
            bound[i] += U * abs(y[i])
    if allowed is not None:
        y[~allowed] = -INF
    return y, bound * 1.01


def adjusted_grad_row(g, x, history, rep, allowed):
    V = g.size
    y = g.copy()
    history = np.asarray(history, dtype=np.int64)
    seen = np.unique(history[(history >= 0) & (history < V)])
    bound = np.zeros(V)
    if rep is not None:
        with np.errstate(all="ignore"):
            y[seen] = np.where(x[seen] > 0, g[seen] / rep, g[seen] * rep)
            bound[seen] = U * np.abs(y[seen]) * 1.01
    if allowed is not None:
        y[~allowed] = 0.0
        bound[~allowed] = 0.0
    return y, bound


def norm(tensors):
    """The norm, scaled so that no square leaves the range of 64 bits."""
    flat = np.concatenate([t.ravel() for t in tensors]) if tensors else np.zeros(0)
    if flat.size == 0:
        return 0.0
    if np.isnan(flat).any():
        return np.nan
    top = np.abs(flat).max()
    if top == 0 or top == INF:
        return float(top)
    return float(np.sqrt(((flat / top) ** 2).sum()) * top)


def close(got, want, bound, what=""):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, what
    odd = ~np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    assert np.array_equal(got[odd & ~np.isnan(want)], want[odd & ~np.isnan(want)]), f"{what}: infinities differ"
    over = np.abs(got[~odd] - want[~odd]) > np.broadcast_to(bound, want.shape)[~odd]
    assert not over.any(), f"{what}: {over.sum()} of {over.size} off, worst {np.abs(got[~odd] - want[~odd])[over].max()}"
