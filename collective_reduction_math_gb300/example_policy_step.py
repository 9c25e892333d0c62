"""One policy-gradient step of a small language model, from its tokens to the
clipped update, with the calls that surround the collectives.

D data-parallel ranks hold a model each, equal on all: a table [V, H] that is
both the embedding and the output head (its rows lie in W shards: rank r has
rows [floor(r*V/W), floor((r+1)*V/W)) as an embedding and the scores of those
columns as a head), and one square layer between the two.  Every step, each
data rank

  1. looks its tokens up, scaled by sqrt(H)                  (mr_embedding);
  2. scores them and applies the penalties and the token mask that the sampler
     used, so that the policy is the one that sampled          (mr_adjust_logits);
  3. takes the log probabilities of the tokens that followed    (mr_logprob);
  4. goes back the same way    (mr_logprob_grad, mr_adjust_logits_grad), the
     embedding's gradient added to the head's               (mr_embedding_grad);

and the gradients are averaged over the data ranks (mr_allreduce) and clipped
together (mr_clip_grad_norm).

    python -m collective_reduction_math_gb300.example_policy_step
"""
from __future__ import annotations


def make_batch(T, V, L, generator):
    """Tokens, the tokens that followed, advantages, and what the sampler applied to each row of scores."""
    import torch
    rand = lambda *shape: torch.rand(*shape, device="cuda", generator=generator)  # noqa: E731
    tokens = (rand(T) ** 3 * V).long()
    tokens[::16] = -1                               # padding
    history = (rand(T, L) ** 3 * V).long()
    n_history = (rand(T) * (L + 1)).long()
    words = (V + 31) // 32
    mask = torch.full((T, words), -1, dtype=torch.int32, device="cuda")
    mask[:, 0] = 0x5555FFFF                         # a few tokens that no row may say
    follow = (rand(T) ** 3 * V).long()
    follow = torch.where((follow < 32) & (follow % 2 == 1) & (follow >= 16), follow - 1, follow)
    follow[tokens < 0] = -1
    return {"tokens": tokens, "follow": follow, "advantage": rand(T) * 2 - 0.5,
            "adjust": {"history": history, "n_history": n_history, "n_prompt": n_history // 2, "repetition": 1.0 + rand(T) * 0.3,
                       "frequency": rand(T) * 0.2, "presence": rand(T) * 0.4, "mask": mask}}


def gradients(table, layer, batch, W, grad_table, grad_layer):
    """Fills both gradients of -mean(advantage * log p(follow)) and returns the log probabilities."""
    import torch

    import collective_reduction_math_gb300 as mr
    V, H = table.shape
    T = batch["tokens"].numel()
    cuts = [r * V // W for r in range(W + 1)]
    rows = lambda t: [t[lo:hi] for lo, hi in zip(cuts, cuts[1:])]  # noqa: E731
    cols = lambda t: [t[:, lo:hi] for lo, hi in zip(cuts, cuts[1:])]  # noqa: E731
    adjust = batch["adjust"]

    x = torch.empty(T, H, device="cuda")
    mr.mr_embedding(rows(table), batch["tokens"], x, scale=H ** 0.5)
    h = torch.tanh(x @ layer)
    scores = h @ table.t()
    policy = torch.empty_like(scores)
    mr.mr_adjust_logits(cols(scores), cols(policy), **adjust)
    logprob, stats = torch.empty(T, device="cuda"), torch.empty(T, 2, device="cuda")
    mr.mr_logprob(cols(policy), batch["follow"], logprob=logprob, stats=stats)

    g = -batch["advantage"] / T
    mr.mr_logprob_grad(cols(policy), batch["follow"], stats, cols(policy), g_logprob=g)
    mr.mr_adjust_logits_grad(cols(scores), cols(policy), cols(policy), **adjust)
    torch.mm(policy.t(), h, out=grad_table)         # the head's part of the table's gradient
    back = (policy @ table) * (1.0 - h * h)
    torch.mm(x.t(), back, out=grad_layer)
    mr.mr_embedding_grad(back @ layer.t(), batch["tokens"], rows(grad_table), scale=H ** 0.5, accumulate=True)
    return logprob


def run(steps=5, D=2, W=3, T=192, V=2003, H=64, L=40, lr=0.2, max_norm=0.05, seed=0, log=print):
    """Returns the norm of each step's gradients before and after clipping."""
    import torch

    import collective_reduction_math_gb300 as mr
    generator = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, device="cuda", generator=generator)  # noqa: E731
    table, layer = normal(V, H) * H ** -0.5 * 0.3, normal(H, H) * H ** -0.5
    models = [(table.clone(), layer.clone()) for _ in range(D)]
    flat = [torch.empty(V * H + H * H, device="cuda") for _ in range(D)]       # each rank's gradients, one behind the other
    norms = []
    for step in range(steps):
        mean = 0.0
        for d in range(D):
            grad_table, grad_layer = flat[d][:V * H].view(V, H), flat[d][V * H:].view(H, H)
            logprob = gradients(*models[d], make_batch(T, V, L, generator), W, grad_table, grad_layer)
            mean += logprob.mean().item() / D
        mr.mr_allreduce(flat, flat, op="avg", algo="auto")
        norm, after = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
        for d in range(D):
            grads = [flat[d][:V * H], flat[d][V * H:]]
            mr.mr_clip_grad_norm(grads, grads, max_norm, norm=norm)
            mr.mr_grad_norm(grads, after)
            for p, g in zip(models[d], grads):
                p -= lr * g.view_as(p)
        norms.append((norm.item(), after.item()))
        log(f"step {step}: mean log probability {mean:.4f}, gradient norm {norms[-1][0]:.4f}, clipped to {norms[-1][1]:.4f}")
    return norms


if __name__ == "__main__":
    run()
