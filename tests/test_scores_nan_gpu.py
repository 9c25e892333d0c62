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


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_masked_places_of_spoilt_rows(mr, dtype, bad):  # noqa: F811
    """All gradients of such a row are NaN: those of masked places, listed or
    not, and of the given token's, too."""
    import torch
    T, V, K, ninf = 6, 3001, 4, float("-inf")
    ids = torch.arange(T, device="cuda")[:, None] * 100 + torch.arange(K, device="cuda") * 7
    x = torch.randn(T, V, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    x[0, 2000] = bad
    x[0, ids[0, 1:3]] = ninf                # masked places in the list
    x[1] = ninf
    x[1, ids[1]] = 1.0
    x[1, ids[1, 1]] = bad                   # nothing left outside the list
    x[2] = ninf
    x[2, ids[2, 0]] = bad                   # nothing else at all
    x[3, ::2] = ninf
    x[3, 1] = bad
    x[4] = ninf
    x[4, 2999] = bad                        # outside the list alone; row 5 stays whole
    x = x.to(_dt(dtype))
    token = ids[:, 1].clone()
    token[3] = 0
    rows, one = Rows(2, T, V, dtype, fill=x), torch.ones(T, device="cuda")

    def check(what, out):
        nan = torch.isnan(torch.cat(out.views, 1).float())
        assert bool(nan[:5].all()) and not bool(nan[5].any()), f"{what}: {nan.sum(1).tolist()} of {V}"
        out.fenced()

    h, st2 = torch.empty(T, device="cuda"), torch.empty(T, 2, device="cuda")
    mr.mr_logprob(rows.views, entropy=h, stats=st2)
    for ent in (None, one):
        out = Rows(2, T, V, dtype)
        mr.mr_logprob_grad(rows.views, token, st2, out.views, g_logprob=one, entropy=h, g_entropy=ent)
        check("log probability", out)
    val = torch.log_softmax(torch.randn(T, K, device="cuda"), 1) - 0.1
    loss, st4 = torch.empty(T, device="cuda"), torch.empty(T, 4, device="cuda")
    for mode in ("renorm", "tail"):
        mr.mr_distill_topk(rows.views, ids, val, loss, stats=st4, mode=mode)
        assert torch.isnan(loss).tolist() == [True] * 5 + [False]
        out = Rows(2, T, V, dtype)
        mr.mr_distill_topk_grad(rows.views, ids, val, st4, one, out.views, mode=mode)
        check(f"gradient, {mode}", out)
        out = Rows(2, T, V, dtype)
        mr.mr_distill_topk_step(rows.views, ids, val, one, loss, out.views, mode=mode)
        check(f"step, {mode}", out)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_teacher_without_mass(mr, dtype):  # noqa: F811
    """Renormalised teacher values that are all -inf: loss and gradient 0, also
    where the student's row is NaN or empty."""
    import torch
    T, V, K = 4, 3001, 4
    ids = torch.arange(T, device="cuda")[:, None] * 100 + torch.arange(K, device="cuda") * 7
    x = torch.randn(T, V, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    x[1, 2000] = float("nan")
    x[2, int(ids[2, 0])] = float("inf")
    x[3] = float("-inf")
    x = x.to(_dt(dtype))
    rows, one = Rows(2, T, V, dtype, fill=x), torch.ones(T, device="cuda")
    val = torch.full((T, K), float("-inf"), device="cuda")
    loss, st = torch.full((T,), 77.0, device="cuda"), torch.empty(T, 4, device="cuda")
    mr.mr_distill_topk(rows.views, ids, val, loss, stats=st)
    assert loss.tolist() == [0.0] * T
    for which in ("gradient", "step"):
        out = Rows(2, T, V, dtype)
        loss.fill_(77.0)
        if which == "gradient":
            mr.mr_distill_topk_grad(rows.views, ids, val, st, one, out.views)
        else:
            mr.mr_distill_topk_step(rows.views, ids, val, one, loss, out.views)
            assert loss.tolist() == [0.0] * T
        assert not torch.cat(out.views, 1).any(), which     # NaN counts as one here
        out.fenced()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("mode", ["renorm", "tail"])
def test_masked_places_of_spoilt_teachers(mr, dtype, mode):  # noqa: F811
    """A column past the vocabulary, or a NaN among the teacher's values, makes
    every gradient of its row NaN, those of masked places too."""
    import torch
    T, V, K, ninf = 4, 3001, 4, float("-inf")
    ids = torch.arange(T, device="cuda")[:, None] * 100 + torch.arange(K, device="cuda") * 7
    x = torch.randn(T, V, device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    x[0, ids[0, 0]] = ninf                  # in the list
    x[1] = ninf
    x[1, ids[1]] = 1.0                      # nothing left outside it
    x[2, ids[2, 3]] = ninf                  # row 3 stays whole
    val = torch.log_softmax(torch.randn(T, K, device="cuda"), 1) - 0.1
    ids[0, 2], ids[1, 2], val[2, 1] = V, V + 5, float("nan")
    x = x.to(_dt(dtype))
    rows, one = Rows(2, T, V, dtype, fill=x), torch.ones(T, device="cuda")
    loss, st = torch.empty(T, device="cuda"), torch.empty(T, 4, device="cuda")
    mr.mr_distill_topk(rows.views, ids, val, loss, stats=st, mode=mode)
    assert torch.isnan(loss).tolist() == [True] * 3 + [False]
    for which in ("gradient", "step"):
        out = Rows(2, T, V, dtype)
        if which == "gradient":
            mr.mr_distill_topk_grad(rows.views, ids, val, st, one, out.views, mode=mode)
        else:
            mr.mr_distill_topk_step(rows.views, ids, val, one, loss, out.views, mode=mode)
        nan = torch.isnan(torch.cat(out.views, 1).float())
        assert bool(nan[:3].all()) and not bool(nan[3].any()), f"{which}: {nan.sum(1).tolist()} of {V}"
        out.fenced()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [1, 40, 3001])
def test_token_past_the_vocabulary_of_an_empty_row(mr, dtype, V):  # noqa: F811
    """NaN, as in any other row; the given token of an empty row otherwise has -inf."""
    import torch
    x = torch.full((3, V), float("-inf"))
    x[2, V // 2] = 1.0
    rows, lp = Rows(1, 3, V, dtype, fill=x.to(_dt(dtype))), torch.empty(3, device="cuda")
    mr.mr_logprob(rows.views, torch.tensor([V, V - 1, V + 7], device="cuda"), logprob=lp)
    assert torch.isnan(lp).tolist() == [True, False, True] and lp[1].item() == float("-inf")
