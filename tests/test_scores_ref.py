"""The 64-bit definitions the score kernels are held against: their gradients
against central differences of their own losses, and the identities that tie
them together (CPU)."""
import numpy as np
import pytest

import score_ref as ref


def _row(rng, n, masked):
    x = rng.normal(0, 2, n)
    if masked:
        x[rng.random(n) < 0.4] = -np.inf
        x[:2] = rng.normal(0, 1, 2)
    return x


def _difference(f, x, direction, h=1e-5):
    return (f(x + h * direction) - f(x - h * direction)) / (2 * h)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("g_lp,g_h", [(1.0, 0.0), (0.0, 1.0), (-0.7, 0.3)])
def test_logprob_gradient_is_the_difference(masked, g_lp, g_h):
    rng = np.random.default_rng(3)
    for n in (2, 5, 40):
        x, token, scale = _row(rng, n, masked), 1, 0.8
        grad = ref.logprob_grad_row(x, token, scale, g_lp, g_h)

        def f(z):
            lp, h, _, _, _ = ref.logprob_row(z, token, scale, 0)
            return g_lp * lp + g_h * h

        for _ in range(3):
            d = rng.normal(0, 1, n)
            # h^2/6 times a third derivative of order 1, and rounding 2^-52 / h
            assert abs(_difference(f, x, d) - (grad * d).sum()) < 1e-7


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("masked", [False, True])
def test_distill_gradient_is_the_difference(masked, tail):
    rng = np.random.default_rng(4)
    for n, k in ((6, 2), (50, 7), (4, 4)):
        x = _row(rng, n, masked and n > 6)
        live = np.nonzero(x > -np.inf)[0]
        ids = rng.permutation(live)[:k]
        val = np.log(rng.dirichlet(np.ones(len(ids))) * 0.9) if tail else rng.normal(0, 1, len(ids))
        if tail and n == k:
            continue                    # the remaining mass would have no place to go
        _, _, grad, _ = ref.distill_row(x, ids, val, 0.8, tail, 1.0, 1.5)
        f = lambda z: 1.5 * ref.distill_row(z, ids, val, 0.8, tail, 1.0, 1.0)[0]  # noqa: E731
        for _ in range(3):
            d = rng.normal(0, 1, n)
            assert abs(_difference(f, x, d) - (grad * d).sum()) < 1e-7


def test_losses_vanish_where_student_is_teacher():
    rng = np.random.default_rng(5)
    x = rng.normal(0, 2, 30)
    lp = ref.log_softmax(x)
    ids = np.argsort(-x)[:6]
    loss, _, grad, _ = ref.distill_row(x, ids, lp[ids], 1.0, True, 1.0, 1.0)
    assert abs(loss) < 1e-12 and np.abs(grad).max() < 1e-12
    ids = np.arange(30)
    loss, _, grad, _ = ref.distill_row(x, ids, x, 1.0, False, 1.0, 1.0)
    assert abs(loss) < 1e-12 and np.abs(grad).max() < 1e-12


def test_rows_with_nothing():
    x = np.full(5, -np.inf)
    lp, h, stats, top, top_lp = ref.logprob_row(x, 2, 1.0, 3)
    assert lp == -np.inf and h == 0 and stats == (-np.inf, 0.0) and top == [0, 1, 2] and top_lp == [-np.inf] * 3
    assert not ref.logprob_grad_row(x, 2, 1.0, 1.0, 1.0).any()
    loss, stats, grad, _ = ref.distill_row(x, np.array([1]), np.array([0.0]), 1.0, False, 1.0, 1.0)
    assert loss == np.inf and not grad.any()
