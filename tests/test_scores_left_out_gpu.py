"""Rows that are left out, in any order and number: the rows beside them come
out with the same bits as when all take part, and what lies in the rows left
out does not matter."""
import numpy as np
import pytest

from test_scores_gpu import Rows, _dt, mr  # noqa: F401  (mr is a fixture)

pytestmark = pytest.mark.gpu


def _out(pattern, T):
    rng = np.random.default_rng(T)
    return {"first": np.arange(T) < 3, "most": rng.random(T) < 0.9, "half": rng.random(T) < 0.5, "last": np.arange(T) >= T - 2,
            "runs": np.arange(T) // 450 % 2 == 1, "all": np.ones(T, bool)}[pattern]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("pattern", ["first", "most", "half", "last", "runs", "all"])
@pytest.mark.parametrize("T,V,W", [(5, 40001, 2), (1900, 20011, 3), (1200, 50257, 1)])
def test_rows_left_out(mr, dtype, pattern, T, V, W):  # noqa: F811
    import torch
    K, k = 40, 7
    out = torch.from_numpy(_out(pattern, T)).cuda()
    x = (torch.randn(T, V, device="cuda", generator=torch.Generator("cuda").manual_seed(V)) * 2).to(_dt(dtype))
    token = torch.arange(T, device="cuda") * 31 % V
    ids = (torch.arange(T, device="cuda")[:, None] * 17 + torch.arange(K, device="cuda") * 101) % V
    val = torch.log_softmax(torch.randn(T, K, device="cuda"), 1) - 0.2
    g = torch.randn(T, device="cuda")

    def run(scores, token, ids):
        rows, r = Rows(W, T, V, dtype, fill=scores), {}
        r["logprob"], r["entropy"], r["stats"] = (torch.full((T,) + s, 77.0, device="cuda") for s in ((), (), (2,)))
        r["top"], r["top_lp"] = torch.full((T, k), 77, dtype=torch.int64, device="cuda"), torch.full((T, k), 77.0, device="cuda")
        mr.mr_logprob(rows.views, token, logprob=r["logprob"], entropy=r["entropy"], stats=r["stats"], top_ids=r["top"],
                      top_logprob=r["top_lp"])
        grads = {n: Rows(W, T, V, dtype) for n in ("logprob_grad", "distill_grad", "step_grad")}
        mr.mr_logprob_grad(rows.views, token, r["stats"], grads["logprob_grad"].views, g_logprob=g, entropy=r["entropy"], g_entropy=g)
        r["loss"], r["loss_stats"], r["step_loss"] = (torch.full((T,) + s, 77.0, device="cuda") for s in ((), (4,), ()))
        mr.mr_distill_topk(rows.views, ids, val, r["loss"], stats=r["loss_stats"], mode="tail")
        mr.mr_distill_topk_grad(rows.views, ids, val, r["loss_stats"], g, grads["distill_grad"].views, mode="tail")
        mr.mr_distill_topk_step(rows.views, ids, val, g, r["step_loss"], grads["step_grad"].views, mode="tail")
        for n, rows_of in grads.items():
            rows_of.fenced()
            r[n] = torch.cat(rows_of.views, 1)
        return r

    whole = run(x, token, ids)
    some = run(torch.where(out[:, None], torch.full_like(x, float("nan")), x), torch.where(out, -1, token),
               torch.where(out[:, None], -1, ids))
    ninf = float("-inf")
    want = {"stats": [ninf, 0.0], "loss_stats": [ninf, 0.0, ninf, 0.0], "top": [-1] * k, "top_lp": [ninf] * k}
    for n, v in some.items():
        assert torch.equal(v[~out], whole[n][~out]), n
        expect = torch.tensor(want.get(n, 0.0), dtype=v.dtype, device="cuda").expand_as(v[out])
        assert torch.equal(v[out], expect), n
