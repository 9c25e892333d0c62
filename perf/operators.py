"""The token-score operators measured: log probabilities of given tokens with
entropy and top alternatives, and distillation from a teacher's top logits,
each forward and backward, over vocabularies that W simulated ranks hold in
shards (rank k has columns [floor(k*V/W), floor((k+1)*V/W))).

`run` computes an operator in its plain form (elementary torch operations in
32 bits, the K teacher values in 64) or, where `own` is true, through
collective_reduction_math_gb300.  `exact` is the definition in 64 bits.
"""
import math

import torch

own = False

# Ops: "logprob" and "distill" are the forward passes, "logprob_grad" and
# "distill_grad" the backward passes from saved statistics, "distill_step" the
# loss and its gradient in one call (the weight of every token's loss is known
# before the call, as in a training step).
OPS = ("logprob", "logprob_grad", "distill", "distill_grad", "distill_step")
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
LEFT_OUT = -100     # the id of a row that is left out (padding)


def _case(name, op, rows, vocab, ranks, dtype, scale=1.0, k=0, tail=False, masked=0.0, pad=0, entropy=True):
    return {"name": name, "op": op, "rows": rows, "vocab": vocab, "ranks": ranks, "dtype": dtype, "scale": scale,
            "k": k, "tail": tail, "masked": masked, "pad": pad, "entropy": entropy}


def listed():
    return [
        # one sequence decoding: the sampled token's log probability and 20 alternatives
        _case("logprob 1 token", "logprob", 1, 131072, 1, "bf16", k=20),
        # a batch of sequences decoding under an output grammar, the vocabulary over 8 ranks
        _case("logprob 48 tokens, masked", "logprob", 48, 128000, 8, "bf16", scale=1.25, k=20, masked=0.75),
        # scoring a short prompt with an odd vocabulary in fp32 (rows that start off any 16-byte boundary)
        _case("logprob prompt fp32 odd", "logprob", 513, 50257, 1, "fp32"),
        # a batch of rollouts scored for a policy gradient
        _case("logprob rollouts", "logprob", 8192, 131072, 4, "bf16"),
        # a teacher scored for its 64 best tokens, from padded rows
        _case("logprob teacher top 64", "logprob", 2048, 160000, 2, "bf16", k=64, pad=64, entropy=False),
        # the policy gradient's backward pass, with an entropy bonus
        _case("logprob grad rollouts", "logprob_grad", 8192, 131072, 4, "bf16"),
        # the same for a small odd fp32 vocabulary, without the bonus
        _case("logprob grad fp32 odd", "logprob_grad", 777, 32003, 3, "fp32", scale=0.8, entropy=False),
        # distillation, evaluation: the loss with a bucket for the teacher's remaining mass
        _case("distill loss", "distill", 4096, 131072, 4, "bf16", k=64, tail=True),
        # the loss of a few short sequences at a temperature, fp32, odd vocabulary
        _case("distill loss fp32 odd", "distill", 37, 50257, 1, "fp32", scale=0.5, k=20),
        # the backward pass after it, 8 ranks, 100 teacher tokens
        _case("distill grad", "distill_grad", 4096, 128000, 8, "bf16", scale=0.5, k=100),
        # a distillation training step over a large batch
        _case("distill step", "distill_step", 8192, 131072, 4, "bf16", k=64, tail=True),
        # a small training step in fp32
        _case("distill step fp32 odd", "distill_step", 301, 65537, 1, "fp32", k=33),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(OPS)
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    vocab = _log_uniform(rng, 8192, 262144)
    if rng.random() < 0.6:
        vocab = vocab // 128 * 128
    # no more bytes than the largest listed case moves
    most = (1 << 30) // (1 if dtype == "bf16" else 2)
    rows = min(_log_uniform(rng, 1, 8192), most // vocab)
    if op.startswith("distill"):
        k = rng.randint(1, 128)
    else:
        k = rng.choice((0, 0, 1, 5, 20, rng.randint(1, 64)))
    return {"op": op, "rows": rows, "vocab": vocab, "ranks": rng.choice((1, 1, 2, 3, 4, 8)), "dtype": dtype,
            "scale": rng.choice((1.0, 1.0, 0.5, 0.7, 1.25, 2.0)), "k": 0 if op == "logprob_grad" else k,
            "tail": rng.random() < 0.5, "masked": rng.choice((0.0, 0.0, 0.0, 0.5, 0.9)),
            "pad": rng.choice((0, 0, 8, 64, 1)), "entropy": rng.random() < 0.7}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _widths(case):
    V, W = case["vocab"], case["ranks"]
    return [(k + 1) * V // W - k * V // W for k in range(W)]


def _left_out(case):
    return case["rows"] // 32


CHUNK = 1 << 27     # elements of fp32 scratch at a time


def _row_chunks(case):
    step = max(1, CHUNK // case["vocab"])
    return [(lo, min(case["rows"], lo + step)) for lo in range(0, case["rows"], step)]


def _shards(case, dtype):
    """W buffers of the rows, `pad` columns wider than the shard."""
    T, pad = case["rows"], case["pad"]
    return [torch.empty(T, w + pad, dtype=dtype, device="cuda")[:, :w] for w in _widths(case)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, V, k = case["rows"], case["vocab"], case["k"]
    dtype, scale = DTYPES[case["dtype"]], case["scale"]
    logits = _shards(case, dtype)
    ids = torch.empty(T, dtype=torch.int64, device="cuda")
    distill = case["op"].startswith("distill")
    t_ids = torch.empty(T, k, dtype=torch.int64, device="cuda") if distill else None
    t_val = torch.empty(T, k, dtype=torch.float32, device="cuda") if distill else None
    stats = torch.empty(T, 4 if distill else 2, device="cuda")
    entropy = torch.empty(T, device="cuda")
    masked = case["masked"]
    for lo, hi in _row_chunks(case):
        # a language model's scores: a broad body, a few tokens well above it
        x = torch.randn(hi - lo, V, device="cuda", generator=g) * 2.0
        hot = torch.randint(0, V, (hi - lo, 16), device="cuda", generator=g)
        boost = torch.rand(hi - lo, 16, device="cuda", generator=g) * 6.0 + 6.0
        if masked:
            x.masked_fill_(torch.rand(hi - lo, V, device="cuda", generator=g) < masked, -math.inf)
        x.scatter_(1, hot, boost)           # so no row is left with nothing
        x = x.to(dtype)
        for s, part in zip(logits, x.split(_widths(case), 1)):
            s[lo:hi].copy_(part)
        # the given tokens: mostly likely ones, never masked
        ids[lo:hi] = hot[:, 0]
        x = x.float()
        if distill:
            # the teacher agrees with the student in part
            t = x.clamp(min=-20.0) * 0.8 + torch.randn(hi - lo, V, device="cuda", generator=g) * 0.7
            t.masked_fill_(x == -math.inf, -30.0)
            v, i = t.topk(k, dim=1)
            if case["tail"]:
                v = v - t.logsumexp(1, keepdim=True)    # the teacher's log probabilities
            t_val[lo:hi], t_ids[lo:hi] = v, i
            rest = x.scatter(1, i, -math.inf)
            stats[lo:hi] = torch.stack(_stats64(x, scale) + _stats64(rest, scale), 1)
        elif case["op"] == "logprob_grad":
            m, s = _stats64(x, scale)
            stats[lo:hi] = torch.stack((m, s), 1)
            y = x.double() * scale
            lp = y - (m.double() + s.double())[:, None]
            entropy[lo:hi] = -(lp.exp() * lp.clamp(min=-1e30)).sum(1)
    out = torch.randperm(T, device="cuda", generator=g)[:_left_out(case)]
    ids[out] = LEFT_OUT
    if distill:
        t_ids[out] = LEFT_OUT
    state = {"case": case, "logits": logits, "ids": ids, "t_ids": t_ids, "t_val": t_val, "stats": stats,
             "entropy": entropy}
    # the loss's weights: advantages, or one over the batch's tokens with a length weighting
    state["g"] = torch.randn(T, device="cuda", generator=g)
    state["g_entropy"] = torch.randn(T, device="cuda", generator=g) * 0.1 if case["entropy"] else None
    # the output buffers such a program keeps
    if case["op"] in ("logprob_grad", "distill_grad", "distill_step"):
        state["grad"] = _shards(case, dtype)
    if case["op"] in ("distill", "distill_step"):
        state["loss"] = torch.empty(T, device="cuda")
    if case["op"] == "distill":
        state["out_stats"] = torch.empty(T, 4, device="cuda")
    if case["op"] == "logprob":
        state["logprob"] = torch.empty(T, device="cuda")
        state["out_entropy"] = torch.empty(T, device="cuda") if case["entropy"] else None
        state["out_stats"] = torch.empty(T, 2, device="cuda")
        state["top_ids"] = torch.empty(T, k, dtype=torch.int64, device="cuda") if k else None
        state["top_logprob"] = torch.empty(T, k, device="cuda") if k else None
    return state


def _stats64(x, scale):
    """The largest scaled score of each row and the log of the sum of exponentials relative to it."""
    m = x.amax(1).mul(scale)
    ref = torch.where(m == -math.inf, torch.zeros_like(m), m)
    s = torch.log((x.double() * scale - ref[:, None].double()).exp().sum(1)).float()
    return m, torch.where(m == -math.inf, torch.zeros_like(s), s)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    op = case["op"]
    if op == "logprob":
        return _logprob(state, case)
    if op == "logprob_grad":
        return _logprob_grad(state, case)
    if op == "distill":
        loss, stats, _ = _distill(state, case, False)
        return {"loss": loss, "stats": stats}
    if op == "distill_grad":
        return {"grad": _distill_grad(state, case)}
    loss, _, grad = _distill(state, case, True)
    return {"loss": loss, "grad": grad}


def _run_own(state, case):
    import collective_reduction_math_gb300 as mr
    op, scale = case["op"], case["scale"]
    if op == "logprob":
        mr.mr_logprob(state["logits"], state["ids"], scale=scale, logprob=state["logprob"],
                      entropy=state["out_entropy"], stats=state["out_stats"], top_ids=state["top_ids"],
                      top_logprob=state["top_logprob"])
        return {"logprob": state["logprob"], "entropy": state["out_entropy"], "stats": state["out_stats"],
                "top_ids": state["top_ids"], "top_logprob": state["top_logprob"]}
    if op == "logprob_grad":
        mr.mr_logprob_grad(state["logits"], state["ids"], state["stats"], state["grad"], g_logprob=state["g"],
                           entropy=state["entropy"], g_entropy=state["g_entropy"], scale=scale)
        return {"grad": state["grad"]}
    kind = "tail" if case["tail"] else "renorm"
    t_scale = 1.0 if case["tail"] else scale
    if op == "distill":
        mr.mr_distill_topk(state["logits"], state["t_ids"], state["t_val"], state["loss"], stats=state["out_stats"],
                           mode=kind, scale=scale, teacher_scale=t_scale)
        return {"loss": state["loss"], "stats": state["out_stats"]}
    if op == "distill_grad":
        mr.mr_distill_topk_grad(state["logits"], state["t_ids"], state["t_val"], state["stats"], state["g"],
                                state["grad"], mode=kind, scale=scale, teacher_scale=t_scale)
        return {"grad": state["grad"]}
    mr.mr_distill_topk_step(state["logits"], state["t_ids"], state["t_val"], state["g"], state["loss"],
                            state["grad"], mode=kind, scale=scale, teacher_scale=t_scale)
    return {"loss": state["loss"], "grad": state["grad"]}


# ---- the plain forms ----

def _softmax_parts(y):
    """Row maximum, log of the sum relative to it, and the shifted scores."""
    m = y.amax(1)
    d = y - torch.where(m == -math.inf, torch.zeros_like(m), m)[:, None]
    s = d.exp().sum(1)
    return m, torch.where(m == -math.inf, torch.zeros_like(m), s.log()), d


def _keep(rows_kept, value, fill):
    shape = (-1,) + (1,) * (value.dim() - 1)
    return torch.where(rows_kept.view(shape), value, torch.full_like(value, fill))


def _logprob(state, case):
    x = torch.cat(state["logits"], 1)
    ids, k = state["ids"], case["k"]
    on = ids >= 0
    y = x.float() * case["scale"]
    m, s, d = _softmax_parts(y)
    lp = d.gather(1, ids.clamp(min=0)[:, None])[:, 0] - s
    out = {"logprob": _keep(on, lp, 0.0), "entropy": None, "top_ids": None, "top_logprob": None,
           "stats": torch.stack((_keep(on, m, -math.inf), _keep(on, s, 0.0)), 1)}
    if case["entropy"]:
        e = d.exp()
        h = s - (e * d.clamp(min=-1e30)).sum(1) / e.sum(1)
        out["entropy"] = _keep(on, h, 0.0)
    if k:
        # one integer a place that orders by value, then by the lower index
        bits = (x.float() + 0.0).view(torch.int32).long()
        key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits) * 2**32 - torch.arange(case["vocab"], device=x.device)
        best = (-(key.topk(k, dim=1).values)) % 2**32
        out["top_ids"] = _keep(on, best, -1)
        out["top_logprob"] = _keep(on, d.gather(1, best) - s[:, None], -math.inf)
    return out


def _logprob_grad(state, case):
    y = torch.cat(state["logits"], 1).float() * case["scale"]
    ids, stats = state["ids"], state["stats"]
    on = ids >= 0
    lp = y - stats[:, :1] - stats[:, 1:]
    p = lp.exp()
    grad = -state["g"][:, None] * p
    if state["g_entropy"] is not None:
        grad = grad - state["g_entropy"][:, None] * p * (lp.clamp(min=-1e30) + state["entropy"][:, None])
    grad.scatter_add_(1, ids.clamp(min=0)[:, None], state["g"][:, None])
    grad = _keep(on, grad * case["scale"], 0.0)
    grad.masked_fill_(y == -math.inf, 0.0)
    return {"grad": list(grad.to(state["logits"][0].dtype).split(_widths(case), 1))}


def _teacher(state, case):
    """log q of the list, q, the remaining mass, and which rows take part."""
    on = (state["t_ids"] >= 0).any(1)
    v = state["t_val"].double()
    if case["tail"]:
        logq = v
        q_rest = (1.0 - logq.exp().sum(1)).clamp(min=0.0)
    else:
        logq = torch.log_softmax(v * case["scale"], 1)
        q_rest = torch.zeros_like(v[:, 0])
    return on, logq.float(), logq.exp().float(), q_rest.float()


def _distill(state, case, with_grad):
    y = torch.cat(state["logits"], 1).float() * case["scale"]
    ids = state["t_ids"].clamp(min=0)
    on, logq, q, q_rest = _teacher(state, case)
    m, s, d = _softmax_parts(y)
    r_m, sr, dr = _softmax_parts(y.scatter(1, ids, -math.inf))
    logp = d.gather(1, ids) - s[:, None]
    loss = (q * (logq - logp)).sum(1)
    log_rest = r_m - m + sr - s
    if case["tail"]:
        loss = loss + torch.where(q_rest > 0, q_rest * (q_rest.log() - log_rest), torch.zeros_like(q_rest))
    stats = torch.stack((_keep(on, m, -math.inf), _keep(on, s, 0.0), _keep(on, r_m, -math.inf), _keep(on, sr, 0.0)), 1)
    grad = None
    if with_grad:
        grad = (dr - sr[:, None]).exp() * (log_rest.exp() - q_rest)[:, None]
        grad = _finish_grad(state, case, grad, ids, logp.exp() - q, on)
    return _keep(on, loss, 0.0), stats, grad


def _finish_grad(state, case, grad, ids, at_list, on):
    grad.scatter_(1, ids, at_list)
    grad = _keep(on, grad * (state["g"] * case["scale"])[:, None], 0.0)
    return list(grad.to(state["logits"][0].dtype).split(_widths(case), 1))


def _distill_grad(state, case):
    y = torch.cat(state["logits"], 1).float() * case["scale"]
    ids, st = state["t_ids"].clamp(min=0), state["stats"]
    on, _, q, q_rest = _teacher(state, case)
    p = (y.gather(1, ids) - st[:, :1] - st[:, 1:2]).exp()
    p_rest = ((st[:, 2] - st[:, 0]) + (st[:, 3] - st[:, 1])).exp()
    grad = (y - st[:, 2:3] - st[:, 3:]).exp() * (p_rest - q_rest)[:, None]
    return _finish_grad(state, case, grad, ids, p - q, on)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    rows = case["rows"] - _left_out(case)
    b = 2 if case["dtype"] == "bf16" else 4
    V, k, T, op = case["vocab"], case["k"], case["rows"], case["op"]
    read = rows * V * b
    if op == "logprob":
        return {"bytes": read + T * (8 + 12 + (4 if case["entropy"] else 0) + 12 * k), "flops": 6.0 * rows * V}
    if op == "logprob_grad":
        return {"bytes": read + T * V * b + T * (8 + 12 + (8 if case["entropy"] else 0)), "flops": 6.0 * rows * V}
    if op == "distill":
        return {"bytes": read + T * (20 + 12 * k), "flops": 4.0 * rows * V}
    return {"bytes": read + T * V * b + T * (24 + 12 * k), "flops": (4.0 if op == "distill_grad" else 7.0) * rows * V}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    op, scale, k = case["op"], case["scale"], case["k"]
    parts = []
    for lo, hi in _row_chunks(dict(case, vocab=4 * case["vocab"])):
        z = torch.cat([s[lo:hi].double() for s in st["logits"]], 1) * scale
        f = {"logprob": _exact_logprob, "logprob_grad": _exact_logprob_grad}.get(op, _exact_distill)
        parts.append(f(case, st, lo, hi, z))
    joined = {n: None if parts[0][n] is None else torch.cat([p[n] for p in parts]) for n in parts[0]}
    if "grad" in joined:
        joined["grad"] = list(joined["grad"].split(_widths(case), 1))
    if op == "logprob" and k == 0:
        joined["top_ids"] = joined["top_logprob"] = None
    names = {"logprob": ("logprob", "entropy", "stats", "top_ids", "top_logprob"), "logprob_grad": ("grad",),
             "distill": ("loss", "stats"), "distill_grad": ("grad",), "distill_step": ("loss", "grad")}[op]
    return {n: joined[n] for n in names}


def _exact_log_softmax(z):
    top = z.max(1, keepdim=True).values
    total = torch.logsumexp(z, 1, keepdim=True)
    return top, total, z - total


def _exact_logprob(case, st, lo, hi, z):
    ids, k = st["ids"][lo:hi], case["k"]
    drop = ids < 0
    top, total, lp = _exact_log_softmax(z)
    got = lp[torch.arange(hi - lo, device=z.device), ids.clamp(min=0)]
    got[drop] = 0.0
    stats = torch.cat((top, total - top), 1)
    stats[drop] = torch.tensor([-math.inf, 0.0], dtype=torch.float64, device=z.device)
    out = {"logprob": got, "entropy": None, "stats": stats, "top_ids": None, "top_logprob": None}
    if case["entropy"]:
        h = torch.special.entr(lp.exp()).sum(1)
        h[drop] = 0.0
        out["entropy"] = h
    if k:
        best = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k].clone()
        chosen = lp.gather(1, best)
        best[drop], chosen[drop] = -1, -math.inf
        out["top_ids"], out["top_logprob"] = best, chosen
    return out


def _exact_logprob_grad(case, st, lo, hi, z):
    # d/dx of g * log p[id] + g_entropy * H, H = -sum p log p
    ids, g = st["ids"][lo:hi], st["g"][lo:hi].double()
    _, _, lp = _exact_log_softmax(z)
    p = lp.exp()
    grad = -p * g[:, None]
    rows = torch.arange(hi - lo, device=z.device)
    grad[rows, ids.clamp(min=0)] += g
    if st["g_entropy"] is not None:
        minus_plogp = torch.special.entr(p)
        grad += st["g_entropy"][lo:hi].double()[:, None] * (minus_plogp - p * minus_plogp.sum(1, keepdim=True))
    grad *= case["scale"]
    grad[ids < 0] = 0.0
    return {"grad": grad}


def _exact_distill(case, st, lo, hi, z):
    ids, v = st["t_ids"][lo:hi], st["t_val"][lo:hi].double()
    drop = ids[:, 0] < 0
    ids = ids.clamp(min=0)
    top, total, lp = _exact_log_softmax(z)
    rest = z.clone()
    rest.scatter_(1, ids, -math.inf)
    r_top, r_total, r_lp = _exact_log_softmax(rest)
    q = v.exp() if case["tail"] else torch.softmax(v * case["scale"], 1)
    logq = v if case["tail"] else torch.log_softmax(v * case["scale"], 1)
    lp_list = lp.gather(1, ids)
    loss = (q * (logq - lp_list)).sum(1)
    p = lp.exp()
    grad = p.clone()
    if case["tail"]:
        q_rest = (1.0 - q.sum(1)).clamp(min=0.0)
        lp_rest = (r_total - total)[:, 0]
        loss = loss + torch.special.xlogy(q_rest, q_rest) - q_rest * lp_rest
        grad = grad - r_lp.exp() * q_rest[:, None]
    grad.scatter_add_(1, ids, -q)
    grad *= (st["g"][lo:hi].double() * case["scale"])[:, None]
    loss[drop], grad[drop] = 0.0, 0.0
    stats = torch.cat((top, total - top, r_top, r_total - r_top), 1)
    stats[drop] = torch.tensor([-math.inf, 0.0] * 2, dtype=torch.float64, device=z.device)
    return {"loss": loss, "grad": grad, "stats": stats}
