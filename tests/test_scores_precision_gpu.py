"""What the distillation's small quantities keep of their precision: the
teacher's masses and what they leave of 1, and the student's probabilities of
listed places.

Tolerances (u = 2^-24): a teacher's mass is the exponential of a given fp32
value as a sum of two floats, off by 2^-33 of itself, and is rounded once, u.
The remaining mass is 1 less the sum of those, so off by 2^-33 (and by its own
rounding).  Probabilities that come out of the row's sums are off by REL of
themselves, as derived in test_scores_gpu.py.
"""
import numpy as np
import pytest

import score_ref as ref
from test_scores_gpu import HALF_STEP, REL, TINY, U, Rows, _close, _run_distill, mr  # noqa: F401  (mr is a fixture)

pytestmark = pytest.mark.gpu


def _step_and_grad(mr, rows, T, V, W, dtype, ids, val, g, stats, **kw):  # noqa: F811
    for which in ("step", "grad"):
        out = Rows(W, T, V, dtype)
        loss, _ = _run_distill(mr, which, rows, out, ids, val, g, stats, **kw)
        yield which, loss, out.host()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("K", [5, 64, 128])
@pytest.mark.parametrize("remainder", [1e-2, 1e-4, 1e-5, 1e-6])
def test_small_remaining_mass(mr, dtype, K, remainder):  # noqa: F811
    """A list that holds nearly all of the teacher's mass, and a student near
    it: the gradient outside the list is softmax * (p_R - q_R)."""
    import torch
    T, V, W = 6, 5000, 2
    rng = np.random.default_rng(K)
    ids = np.stack([rng.permutation(V)[:K] for _ in range(T)]).astype(np.int64)
    q = rng.gamma(0.3, 1.0, (T, K)) + 1e-9
    val = np.log(q / q.sum(1, keepdims=True) * (1 - remainder)).astype(np.float32)
    x = np.log(1.5 * remainder / V) + rng.normal(0, 1, (T, V))
    np.put_along_axis(x, ids, val + rng.normal(0, 0.05, (T, K)), 1)
    x = torch.from_numpy(x).to(torch.float32 if dtype == "fp32" else torch.bfloat16)
    xs, g = x.double().numpy(), rng.normal(0, 1, T).astype(np.float32)
    res = [ref.distill_row(xs[t], ids[t], val[t].astype(np.float64), 1.0, True, 1.0, float(g[t])) for t in range(T)]
    stats = np.array([r[1] for r in res])
    rows = Rows(W, T, V, dtype, fill=x)
    for which, loss, grad in _step_and_grad(mr, rows, T, V, W, dtype, ids, val, g, stats.astype(np.float32), mode="tail"):
        for t in range(T):
            m, s, m_r, s_r = stats[t]
            p, p_rest = np.exp(xs[t] - m - s), np.exp(m_r - m + s_r - s)
            q_t = np.exp(val[t].astype(np.float64))
            q_rest = max(0.0, 1 - q_t.sum())
            parts = np.exp(xs[t] - m_r - s_r) * (2 * REL * (p_rest + q_rest) + 2.0 ** -32)
            parts[ids[t]] = 2 * REL * p[ids[t]] + 4 * U * q_t
            parts *= abs(g[t])
            _close(grad[t], res[t][2], parts + HALF_STEP[dtype] * (np.abs(res[t][2]) + parts) + TINY[dtype], f"{which} row {t}")
            if which == "step":
                _close(loss[t], res[t][0], 2 * REL * res[t][3] + 2.0 ** -32 * (abs(np.log(max(q_rest, 2.0 ** -33))) + abs(np.log(p_rest))))


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("K", [1, 5, 33, 64, 100, 128])
def test_masses_are_rounded_once(mr, K, tail):  # noqa: F811
    """Listed places that the student gives next to nothing: their gradient is
    -q, which is off by its rounding alone."""
    import torch
    T, V = 4, 700
    rng = np.random.default_rng(K)
    ids = np.stack([rng.permutation(V)[:K] for _ in range(T)]).astype(np.int64)
    t_scale = float(np.float32(1.0 if tail else 0.7))
    val = rng.normal(0, 3, (T, K))
    if tail:
        val -= np.log(np.exp(val).sum(1, keepdims=True)) + 0.05
    val = val.astype(np.float32)
    x = np.full((T, V), 1.0)
    np.put_along_axis(x, ids, -150.0, 1)        # p < 2^-200: nothing beside q
    rows = Rows(1, T, V, "fp32", fill=torch.from_numpy(x).float())
    stats = np.array([ref.distill_row(x[t], ids[t], val[t].astype(np.float64), 1.0, tail, t_scale, 1.0)[1] for t in range(T)])
    for which, _, grad in _step_and_grad(mr, rows, T, V, 1, "fp32", ids, val, np.ones(T, np.float32), stats.astype(np.float32),
                                         mode="tail" if tail else "renorm", teacher_scale=t_scale):
        for t in range(T):
            q = ref.teacher(val[t].astype(np.float64), tail, t_scale)[1]
            _close(grad[t][ids[t]], -q, q * (U + 2.0 ** -31) + TINY["fp32"], f"{which} row {t}")


@pytest.mark.parametrize("K", [20, 128])
def test_listed_probabilities_far_below_the_best(mr, K):  # noqa: F811
    """Listed places without a teacher's mass, of scores down to 60 below the
    row's only large one: their gradient is p.  The difference from the best
    score is exact here, and so is the row's sum but for u; the exponential is
    off by 2^-22, by the rounding of the log sum that the gradient is given
    (u, of e^-60 and less here) and by that of its argument's last step."""
    import torch
    T, V = 4, 1500
    rng = np.random.default_rng(K)
    ids = np.stack([1 + rng.permutation(V - 1)[:K] for _ in range(T)]).astype(np.int64)
    x = np.full((T, V), -64.0)
    x[:, 0] = 0.0
    np.put_along_axis(x, ids, -np.round(rng.uniform(20, 60, (T, K)) * 4096) / 4096, 1)
    val = np.full((T, K), -np.inf, np.float32)
    val[:, 0] = 0.0
    rows = Rows(1, T, V, "fp32", fill=torch.from_numpy(x).float())
    res = [ref.distill_row(x[t], ids[t], val[t].astype(np.float64), 1.0, False, 1.0, 1.0) for t in range(T)]
    stats = np.array([r[1] for r in res])
    for which, _, grad in _step_and_grad(mr, rows, T, V, 1, "fp32", ids, val, np.ones(T, np.float32), stats.astype(np.float32),
                                         mode="renorm"):
        for t in range(T):
            want = res[t][2][ids[t][1:]]
            _close(grad[t][ids[t][1:]], want, np.abs(want) * (2.0 ** -22 + 4 * U), f"{which} row {t}")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V,K", [(4000, 20), (4000, 128), (20, 20), (64, 64)])
def test_list_of_all_that_is_left(mr, dtype, V, K):  # noqa: F811
    """Teacher and student under one mask that leaves at most K places, the list
    from mr_logprob: what its log probabilities lack of 1 is their rounding,
    and the loss is finite.  A list that leaves a real remainder is +inf."""
    import torch
    T, k = 60, min(K, 64)
    rng = np.random.default_rng(V + K)
    x, teacher = rng.normal(0, 3, (2, T, V))
    for t in range(T):
        if V > K:
            left = rng.permutation(V)[:1 + t % k]
            mask = np.ones(V, bool)
            mask[left] = False
            x[t, mask] = teacher[t, mask] = -np.inf
    dt = torch.float32 if dtype == "fp32" else torch.bfloat16
    x, teacher = torch.from_numpy(x).to(dt), torch.from_numpy(teacher).to(dt)
    ids = torch.full((T, K), -1, dtype=torch.int64, device="cuda")
    val = torch.zeros(T, K, device="cuda")
    top, top_lp = torch.empty(T, k, dtype=torch.int64, device="cuda"), torch.empty(T, k, device="cuda")
    mr.mr_logprob(Rows(2, T, V, dtype, fill=teacher).views, top_ids=top, top_logprob=top_lp)
    ids[:, :k], val[:, :k] = top, top_lp
    ids, val = ids.cpu().numpy(), val.cpu().numpy()
    xs, rows = x.double().numpy(), Rows(2, T, V, dtype, fill=x)
    g = np.ones(T, np.float32)
    want, size, lacks = np.zeros(T), np.zeros(T), []
    for t in range(T):
        q = np.exp(val[t, :k].astype(np.float64))
        on, lp = q > 0, ref.log_softmax(xs[t])
        terms = q[on] * (val[t, :k].astype(np.float64)[on] - lp[ids[t, :k]][on])
        want[t], size[t] = terms.sum(), (q[on] * (np.abs(val[t, :k][on]) + np.abs(lp[ids[t, :k]][on]) + 1)).sum()
        lacks.append(1 - q.sum())
    assert max(lacks) > 0 and np.abs(lacks).max() < 2.0 ** -18
    for which in ("forward", "step"):
        loss, _ = _run_distill(mr, which, rows, Rows(2, T, V, dtype), ids, val, g, None, mode="tail")
        _close(loss, want, 2 * REL * size, which)
    low = np.where(val > -np.inf, val - np.float32(0.01), val)
    for which in ("forward", "step"):
        loss, _ = _run_distill(mr, which, rows, Rows(2, T, V, dtype), ids, low, g, None, mode="tail")
        assert (loss == np.inf).all(), which
