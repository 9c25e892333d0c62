"""Rows of scores that hold one NaN or +inf: every output of the row is NaN,
wherever in the row it lies and whatever the same thread sees after it."""
import numpy as np
import pytest

from test_scores_gpu import Rows, _dt, mr  # noqa: F401  (mr is a fixture)

pytestmark = pytest.mark.gpu


def _rows_with_one(T, V, W, dtype, seed):
    """Scores on the GPU, and which rows are spoilt.  Row t has a NaN, a +inf,
    or a +inf before a NaN at a place of its own; in every other such row the
    places after it are masked, all of them or only the next 40000 bytes (a
    superblock for each warp of a CTA, and more).  Every 5th row stays whole."""
    import torch
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(T, V, device="cuda", generator=g) * 2
    rng = np.random.default_rng(seed)
    spoilt = np.arange(T) % 5 != 4
    for t in range(T):
        if not spoilt[t]:
            continue
        at = int(rng.integers(0, V))
        if t % 3 == 0:      # a round of superblocks (8 warps of 2 KiB) before the row's last, by a lane past the row's end
            sb = 2048 // (4 if dtype == "fp32" else 2)
            last = (V - 1) // sb
            at = max(0, last - 8) * sb + min(sb - 1, (V - 1) % sb + 20)
            at = min(at, V - 1)
        if t % 2:
            x[t, at + 1: V if t % 4 == 1 else at + 40000 // (4 if dtype == "fp32" else 2)] = float("-inf")
        x[t, at] = float("inf") if t % 7 == 3 else float("nan")
        if t % 7 == 5:
            x[t, at // 2] = float("inf")
    return x.to(_dt(dtype)), spoilt


# T: rows on wide clusters, on small ones, and several rows a CTA
SHAPES = [(1, 50257, 1), (6, 50257, 1), (6, 200003, 3), (97, 50257, 1), (97, 32003, 3), (1200, 50257, 1), (1200, 9001, 2)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T,V,W", SHAPES)
def test_one_nan_reaches_every_output(mr, dtype, T, V, W):  # noqa: F811
    import torch
    x, spoilt = _rows_with_one(T, V, W, dtype, T + V)
    rows = Rows(W, T, V, dtype, 0, 0, x)
    ids = torch.arange(T, device="cuda") * 7 % V
    k = 5

    def outputs(*shape):
        return torch.full((T,) + shape, 77.0, device="cuda")

    def check(what, value, at=None):
        wrong = torch.isnan(value.reshape(T, -1).float()) != torch.from_numpy(spoilt).cuda()[:, None]
        if at is not None:
            wrong &= at
        assert not bool(wrong.any()), f"{what}: rows {sorted(set(wrong.nonzero()[:, 0].tolist()))[:8]}"

    for top in (0, k):
        lp, h, stats, top_lp = outputs(), outputs(), outputs(2), outputs(k)
        mr.mr_logprob(rows.views, ids, logprob=lp, entropy=h, stats=stats, top_logprob=top_lp if top else None)
        live = x.gather(1, ids[:, None])[:, 0] != float("-inf")
        for what, v in (("logprob", lp), ("entropy", h), ("stats", stats)) + ((("top", top_lp),) if top else ()):
            check(f"{what}, top {top}", v)
        assert bool(torch.isfinite(lp[live & ~torch.from_numpy(spoilt).cuda()]).all())
        lp2 = outputs()
        mr.mr_logprob(rows.views, ids, logprob=lp2)         # without the entropy's sums
        check("logprob alone", lp2)

    t_ids = (torch.arange(T, device="cuda")[:, None] * 11 + torch.arange(k, device="cuda") * 13) % V
    t_val = torch.log_softmax(torch.randn(T, k, device="cuda"), 1) - 0.1
    weight = torch.ones(T, device="cuda")
    unmasked = x != float("-inf")
    for mode in ("renorm", "tail"):
        loss, st, loss2, out = outputs(), outputs(4), outputs(), Rows(W, T, V, dtype)
        mr.mr_distill_topk(rows.views, t_ids, t_val, loss, stats=st, mode=mode)
        check("loss", loss)
        check("row's statistics", st[:, :2])
        mr.mr_distill_topk_step(rows.views, t_ids, t_val, weight, loss2, out.views, mode=mode)
        check("step's loss", loss2)
        check("step's gradient", torch.cat(out.views, 1), unmasked)
        out = Rows(W, T, V, dtype)
        mr.mr_distill_topk_grad(rows.views, t_ids, t_val, st, weight, out.views, mode=mode)
        check("gradient", torch.cat(out.views, 1), unmasked)
        out.fenced()
