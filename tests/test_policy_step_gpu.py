"""The embedding, the adjusted scores, the token scores, the all-reduce and the
clipping in the order of a training step (example_policy_step), its gradients
against the same step's in 64 bits by automatic differentiation; and a decoding
step of single tokens, captured into a graph."""
import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
REL = 2.0 ** -16        # of a probability by the token scores (derived at the head of test_scores_gpu.py)


@pytest.fixture(scope="module")
def mr():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import __graft_entry__
    __graft_entry__.build()
    import collective_reduction_math_gb300 as m
    m.load()
    return m


def _adjusted64(scores, batch):
    """The adjusted scores in 64 bits, differentiable."""
    import torch
    a = {k: v.cpu() for k, v in batch["adjust"].items()}
    T, V = scores.shape
    at = torch.arange(a["history"].shape[1])
    there = at < a["n_history"][:, None]
    said = there & (at >= a["n_prompt"][:, None])
    seen = torch.zeros(T, V).scatter_add_(1, a["history"], there.float()) > 0
    times = torch.zeros(T, V, dtype=torch.float64).scatter_add_(1, a["history"], said.double())
    rep = a["repetition"].double()[:, None]
    y = torch.where(seen, torch.where(scores > 0, scores / rep, scores * rep), scores)
    y = y - a["frequency"].double()[:, None] * times - a["presence"].double()[:, None] * (times > 0)
    bits = (a["mask"].long()[:, :, None] >> torch.arange(32)) & 1
    return y.masked_fill(bits.view(T, -1)[:, :V] == 0, float("-inf"))


@pytest.mark.parametrize("W", [1, 3])
def test_gradients_of_the_step(mr, W):
    import torch
    from collective_reduction_math_gb300 import example_policy_step as ex
    T, V, H, L = 96, 1003, 32, 24
    gen = torch.Generator(device="cuda").manual_seed(1)
    table = torch.randn(V, H, device="cuda", generator=gen) * H ** -0.5 * 0.3
    layer = torch.randn(H, H, device="cuda", generator=gen) * H ** -0.5
    batch = ex.make_batch(T, V, L, gen)
    grad_table, grad_layer = torch.empty_like(table), torch.empty_like(layer)
    logprob = ex.gradients(table, layer, batch, W, grad_table, grad_layer)

    w, m = table.double().cpu().requires_grad_(), layer.double().cpu().requires_grad_()
    tokens, follow = batch["tokens"].cpu(), batch["follow"].cpu()
    on = tokens >= 0
    x = w[tokens.clamp(min=0)] * H ** 0.5 * on[:, None]
    h = torch.tanh(x @ m)
    scores = h @ w.t()
    lp = torch.log_softmax(_adjusted64(scores, batch), 1)
    got = lp[torch.arange(T), follow.clamp(min=0)] * on
    (-(batch["advantage"].double().cpu() * got).mean()).backward()

    # What fp32 may do.  A score is a sum of H products of a row h that is itself the tanh (off by 4 U at most) of a sum
    # of H products of looked-up values: off by delta; its adjustment adds 4 roundings of values no larger than `top`.
    with torch.no_grad():
        size = lambda a, b: a.abs() @ b.abs()  # noqa: E731
        dh = (H + 6) * U * size(x, m) + 4 * U
        top = scores.abs().max() * 1.4 + 2
        delta = float((dh @ w.abs().t() + (H + 2) * U * size(h, w.t())).max() * 1.4 + 4 * U * top)
        wrong = REL + 4 * delta + 8 * U         # relative, of each probability and of what follows from it
        lp, got = lp.detach(), got.detach()
        p = lp.exp()
        one = torch.zeros(T, V, dtype=torch.float64)
        one[torch.arange(T)[on], follow[on]] = 1.0
        dscore = (batch["advantage"].double().cpu().abs() / T * on)[:, None] * (p + one) * 1.4     # its terms' magnitudes
        back = dscore @ w.abs()
        # d tanh = 1 - h^2, off by 2 |h| dh; sums of V, H and T products, each off by its length times U
        loss_of = wrong + (V + H + T + 8) * U
        head = dscore.t() @ h.abs() * (loss_of + float((dh / h.abs().clamp(min=1e-3)).max()))
        dx = (back * (loss_of + 2 * float(dh.max()))) @ m.abs().t()
        embed = torch.zeros_like(w).index_add_(0, tokens[on], dx[on] * H ** 0.5)
        layer_bound = x.abs().t() @ (back * (loss_of + 2 * float(dh.max())))
    assert float((logprob.double().cpu() - got).abs().max()) <= REL + 4 * delta + 8 * U * float(lp[lp > -1e30].abs().max())
    assert bool(((grad_table.double().cpu() - w.grad).abs() <= head + embed + 4 * U * w.grad.abs()).all())
    assert bool(((grad_layer.double().cpu() - m.grad).abs() <= layer_bound).all())
    # the bounds say something: most gradients are far larger
    assert float((head + embed).norm()) < 0.05 * float(w.grad.norm())


def test_the_example_runs(mr):
    from collective_reduction_math_gb300 import example_policy_step as ex
    before = mr.mr_launch_count()
    lines = []
    norms = ex.run(steps=3, T=64, V=501, H=32, L=12, log=lines.append)
    assert mr.mr_launch_count() - before >= 3 * (2 * 8 + 1 + 2 * 4)
    assert len(lines) == 3
    for norm, after in norms:
        # the factor and each product are off by the norm's 34 U and two roundings, the second norm by its own 34 U
        assert norm > 0 and after <= min(norm, 0.05) * (1 + 72 * U)


def test_a_decoding_step_in_a_graph(mr):
    """Single tokens: lookup, adjusted scores in place, log probability and alternatives, replayed with other tokens."""
    import torch
    V, H, L = 8009, 128, 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    table = (torch.randn(V, H, device="cuda", generator=gen) * 0.1).bfloat16()
    token = torch.tensor([5], device="cuda")
    history = torch.randint(0, V, (1, L), device="cuda", generator=gen)
    length = torch.tensor([3], device="cuda")
    rep = torch.tensor([1.25], device="cuda")
    x, scores = torch.empty(1, H, dtype=torch.bfloat16, device="cuda"), torch.empty(1, V, dtype=torch.bfloat16, device="cuda")
    top, top_lp = torch.empty(1, 5, dtype=torch.int64, device="cuda"), torch.empty(1, 5, device="cuda")

    def step():
        mr.mr_embedding([table], token, x, scale=4.0)
        torch.mm(x, table.t(), out=scores)
        mr.mr_adjust_logits([scores], [scores], history=history, n_history=length, repetition=rep)
        mr.mr_logprob([scores], top_ids=top, top_logprob=top_lp)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(6):
        token.fill_(17 * k + 1)
        history[0, length] = token          # what was said last
        length += 1
        graph.replay()
        torch.cuda.synchronize()
        got, got_lp = top.clone(), top_lp.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, top) and torch.equal(got_lp, top_lp)
        want = (table[token].float() * 4.0).bfloat16()
        assert torch.equal(x, want)
        y = (want @ table.t()).float()[0]
        seen = history[0, :int(length)].unique()
        y[seen] = torch.where(y[seen] > 0, y[seen] / 1.25, y[seen] * 1.25)
        assert torch.equal(scores[0], y.bfloat16())
        assert float(scores[0][top[0, 0]]) == float(scores.max())
