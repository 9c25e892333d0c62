"""The token-score operators and the collectives in one training loop.

D data-parallel ranks train one output head [V, H], whose vocabulary lies in W
shards (rank r has rows [floor(r*V/W), floor((r+1)*V/W))).  Every step, each
data rank

  1. scores its tokens with the teacher and keeps the teacher's best K log
     probabilities (mr_logprob);
  2. computes the distillation loss and its gradient, in place of the student's
     scores (mr_distill_topk_step);
  3. scores the tokens it sampled and adds the policy gradient with an entropy
     bonus (mr_logprob, mr_logprob_grad);

and the head's gradients are averaged over the data ranks (mr_allreduce).

    python -m collective_reduction_math_gb300.example_post_training
"""
from __future__ import annotations


def run(steps=20, D=2, W=4, T=256, V=8000, H=64, K=32, lr=60.0, seed=0, log=print):
    """Returns the mean distillation loss of each step."""
    import torch

    import collective_reduction_math_gb300 as mr

    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, device="cuda", generator=g)  # noqa: E731
    cuts = [r * V // W for r in range(W + 1)]
    teacher = [normal(cuts[r + 1] - cuts[r], H) * 0.4 for r in range(W)]
    # one head per data rank, equal on all; its shards lie one behind the other
    heads = [torch.zeros(V, H, device="cuda") for _ in range(D)]
    grads = [torch.empty(V, H, device="cuda") for _ in range(D)]
    weight = torch.full((T,), 1.0 / T, device="cuda")
    losses = []
    for step in range(steps):
        mean_loss = 0.0
        for d in range(D):
            h = normal(T, H)
            scores = lambda head: [(h @ w.t()).bfloat16() for w in head]  # noqa: E731
            head = [heads[d][cuts[r]:cuts[r + 1]] for r in range(W)]

            # the teacher's best K log probabilities
            top_ids = torch.empty(T, K, dtype=torch.int64, device="cuda")
            top_logprob = torch.empty(T, K, device="cuda")
            mr.mr_logprob(scores(teacher), top_ids=top_ids, top_logprob=top_logprob)

            # loss and gradient, in place
            x = scores(head)
            loss = torch.empty(T, device="cuda")
            mr.mr_distill_topk_step(x, top_ids, top_logprob, weight, loss, x, mode="tail")
            for r in range(W):
                grads[d][cuts[r]:cuts[r + 1]] = x[r].float().t() @ h
            mean_loss += loss.mean().item() / D

            # a policy gradient on sampled tokens: raise what the teacher likes
            x = scores(head)
            token = top_ids[torch.arange(T, device="cuda"), torch.randint(0, K, (T,), device="cuda", generator=g)]
            logprob, entropy = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
            stats = torch.empty(T, 2, device="cuda")
            mr.mr_logprob(x, token, logprob=logprob, entropy=entropy, stats=stats)
            advantage = top_logprob.exp().gather(1, (top_ids == token[:, None]).int().argmax(1, keepdim=True))[:, 0]
            bonus = torch.full((T,), -1e-3 / T, device="cuda")
            mr.mr_logprob_grad(x, token, stats, x, g_logprob=-0.1 * advantage / T, entropy=entropy, g_entropy=bonus)
            for r in range(W):
                grads[d][cuts[r]:cuts[r + 1]] += x[r].float().t() @ h

        mr.mr_allreduce([t.view(-1) for t in grads], [t.view(-1) for t in grads], op="avg", algo="auto")
        for d in range(D):
            heads[d] -= lr * grads[d]
        losses.append(mean_loss)
        log(f"step {step}: distillation loss {mean_loss:.4f}, entropy {entropy.mean().item():.3f}, "
            f"log probability of the sampled tokens {logprob.mean().item():.3f}")
    return losses


if __name__ == "__main__":
    run()
