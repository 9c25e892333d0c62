"""The operators at both ends of a policy's step measured: the embedding lookup
and its gradient by sorted tokens (a table whose rows W simulated ranks hold in
shards), penalties, biases and token masks on the scores (whose columns they
hold in shards), each forward and backward, and the norm of many gradients with
their clipping.  Rank r of W has rows or columns [floor(r*V/W), floor((r+1)*V/W)).

`run` computes an operator in its plain form (elementary torch operations in
32 bits, long sums in 64) or, where `own` is true, through
collective_reduction_math_gb300.  `exact` is the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

OPS = ("embed", "embed_grad", "adjust", "adjust_grad", "norm", "clip")
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}
LEFT_OUT = -100     # the id of a position that is left out (padding)


def _embed(name, rows, vocab, hidden, ranks, dtype, scale=1.0):
    return {"name": name, "op": "embed", "rows": rows, "vocab": vocab, "hidden": hidden, "ranks": ranks, "dtype": dtype,
            "scale": scale}


def _embed_grad(name, rows, vocab, hidden, ranks, dtype, table, accumulate, scale=1.0):
    return {"name": name, "op": "embed_grad", "rows": rows, "vocab": vocab, "hidden": hidden, "ranks": ranks,
            "dtype": dtype, "table": table, "accumulate": accumulate, "scale": scale}


def _adjust(name, op, rows, vocab, ranks, dtype, history, bias=0, masked=0.0):
    return {"name": name, "op": op, "rows": rows, "vocab": vocab, "ranks": ranks, "dtype": dtype, "history": history,
            "bias": bias, "masked": masked}


def _tensors(name, op, tensors, elements, dtype, norm=4.0):
    return {"name": name, "op": op, "tensors": tensors, "elements": elements, "dtype": dtype, "norm": norm}


def listed():
    return [
        # one sequence decoding: the token that was sampled last
        _embed("embed 1 token", 1, 131072, 8192, 1, "bf16"),
        # the batch of a training step, its table over 4 ranks, scaled by sqrt(hidden)
        _embed("embed batch", 32768, 131072, 8192, 4, "bf16", scale=8192.0 ** 0.5),
        # a fine-tuning step on a few sequences: fp32, odd vocabulary and row length, every row of the gradient written
        _embed_grad("embed grad fp32 odd", 777, 32003, 1001, 3, "fp32", "fp32", False),
        # a micro-batch, added to the fp32 gradient that it shares with the output head
        _embed_grad("embed grad batch", 16384, 131072, 4096, 4, "bf16", "fp32", True, scale=64.0),
        # one sequence decoding under a grammar, with penalties on what it has said
        _adjust("adjust 1 row", "adjust", 1, 131072, 1, "bf16", 1500, bias=16, masked=0.75),
        # a batch of rollouts scored with the penalties that they were sampled with
        _adjust("adjust rollouts", "adjust", 4096, 131072, 4, "bf16", 2048, bias=16, masked=0.25),
        # the gradient of a few rows, fp32, odd vocabulary (rows off any 16-byte boundary)
        _adjust("adjust grad fp32 odd", "adjust_grad", 37, 50257, 3, "fp32", 700),
        # the policy gradient's way back through the penalties
        _adjust("adjust grad rollouts", "adjust_grad", 4096, 131072, 4, "bf16", 2048, masked=0.25),
        # an adapter's gradients
        _tensors("norm of an adapter", "norm", 24, 1 << 20, "fp32"),
        # a model's bf16 gradients, or a rank's part of a larger one's
        _tensors("norm of a model", "norm", 290, 1500000000, "bf16"),
        # a 25 MiB bucket's worth of mixed tensors
        _tensors("clip a bucket", "clip", 40, 9000000, "mixed"),
        # a model's gradients clipped, into the buffers that the optimizer reads
        _tensors("clip a model", "clip", 290, 700000000, "mixed"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(OPS)
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    ranks = rng.choice((1, 1, 2, 3, 4, 8))
    vocab = _log_uniform(rng, 8192, 262144)
    if rng.random() < 0.6:
        vocab = vocab // 128 * 128
    if op in ("embed", "embed_grad"):
        hidden = _log_uniform(rng, 128, 8192)
        if rng.random() < 0.7:
            hidden = hidden // 64 * 64
        # the table and the rows in no more bytes than the largest listed cases'
        vocab = min(vocab, (1 << 29) // hidden)
        rows = min(_log_uniform(rng, 1, 32768), (1 << 28) // hidden // (1 if dtype == "bf16" else 2))
        scale = rng.choice((1.0, 1.0, 0.5, hidden ** 0.5))
        if op == "embed":
            return {"op": op, "rows": rows, "vocab": vocab, "hidden": hidden, "ranks": ranks, "dtype": dtype, "scale": scale}
        return {"op": op, "rows": rows, "vocab": vocab, "hidden": hidden, "ranks": ranks, "dtype": dtype,
                "table": rng.choice(("fp32", dtype)), "accumulate": rng.random() < 0.5, "scale": scale}
    if op in ("adjust", "adjust_grad"):
        most = (1 << 29) // (1 if dtype == "bf16" else 2)
        history = rng.choice((0, _log_uniform(rng, 1, 4096), _log_uniform(rng, 64, 4096)))
        bias = rng.choice((0, 0, 1, rng.randint(2, 300))) if op == "adjust" else 0
        return {"op": op, "rows": min(_log_uniform(rng, 1, 4096), most // vocab), "vocab": vocab, "ranks": ranks,
                "dtype": dtype, "history": history, "bias": bias,
                "masked": rng.choice((0.0, 0.1, 0.75, 0.99) if history or bias else (0.1, 0.75, 0.99))}
    tensors, dtype = _log_uniform(rng, 1, 600), rng.choice((dtype, "mixed"))
    most = (1850000000 if op == "clip" else 3000000000) // BYTES.get(dtype, 4)      # bytes, the larger type's where mixed
    return {"op": op, "tensors": tensors, "elements": max(tensors, _log_uniform(rng, 1000, most)), "dtype": dtype,
            "norm": rng.choice((0.5, 4.0, 40.0))}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _cuts(V, W):
    return [r * V // W for r in range(W + 1)]


def _shards(t, W, dim):
    """W slices of one buffer along `dim`, as the simulated ranks hold them."""
    cuts = _cuts(t.shape[dim], W)
    return [t.narrow(dim, lo, hi - lo) for lo, hi in zip(cuts, cuts[1:])]


def _token_weights(V):
    """How often the tokens of a vocabulary occur: few often, most hardly ever."""
    w = 1.0 / (np.arange(V) + 3.0)
    return w / w.sum()


def _tokens(shape, V, g):
    edges = torch.from_numpy(np.cumsum(_token_weights(V))).cuda()
    u = torch.rand(shape, device="cuda", dtype=torch.float64, generator=g)
    return torch.searchsorted(edges, u).clamp(max=V - 1)


def _left_out(case):
    return case["rows"] // 32


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] in ("embed", "embed_grad"):
        return _prepare_embedding(case, g)
    if case["op"] in ("adjust", "adjust_grad"):
        return _prepare_adjust(case, g)
    return _prepare_tensors(case, g)


def _prepare_embedding(case, g):
    T, V, H, W, dtype = case["rows"], case["vocab"], case["hidden"], case["ranks"], DTYPES[case["dtype"]]
    ids = _tokens((T,), V, g)
    ids[torch.randperm(T, device="cuda", generator=g)[:_left_out(case)]] = LEFT_OUT
    state = {"case": case, "ids": ids}
    if case["op"] == "embed":
        state["table"] = torch.empty(V, H, dtype=dtype, device="cuda").normal_(0.0, 0.02, generator=g)
        state["shards"] = _shards(state["table"], W, 0)
        state["out"] = torch.empty(T, H, dtype=dtype, device="cuda")
    else:
        state["g"] = torch.empty(T, H, dtype=dtype, device="cuda").normal_(0.0, 0.01, generator=g)
        state["table"] = torch.empty(V, H, dtype=DTYPES[case["table"]], device="cuda")
        if case["accumulate"]:      # what earlier calls left there
            state["table"].normal_(0.0, 0.01, generator=g)
        state["shards"] = _shards(state["table"], W, 0)
    return state


def _prepare_adjust(case, g):
    T, V, W, L, K, dtype = (case[n] for n in ("rows", "vocab", "ranks", "history", "bias", "dtype"))
    x = torch.empty(T, V, dtype=DTYPES[dtype], device="cuda").normal_(0.0, 2.5, generator=g)
    state = {"case": case, "x": x, "logits": _shards(x, W, 1), "history": None, "n_history": None, "n_prompt": None,
             "repetition": None, "frequency": None, "presence": None, "bias_ids": None, "bias": None, "mask": None}
    rand = lambda *shape: torch.rand(*shape, device="cuda", generator=g)  # noqa: E731
    if L:
        # sequences of different lengths, a prompt at the front of each; the model repeats some of what stands there
        state["history"] = _tokens((T, L), V, g)
        state["n_history"] = ((0.5 + 0.5 * rand(T)) * L).ceil().long()
        state["n_prompt"] = (rand(T) * 0.5 * state["n_history"]).long()
        state["repetition"] = 1.0 + 0.3 * rand(T)
        state["frequency"] = 0.2 * rand(T)
        state["presence"] = 0.5 * rand(T)
    if K:
        state["bias_ids"] = torch.randperm(V, device="cuda", generator=g)[:K].repeat(T, 1)
        state["bias"] = torch.randn(T, K, device="cuda", generator=g) * 3.0
    if case["masked"]:
        words = torch.zeros(T, (V + 31) // 32, dtype=torch.int32, device="cuda")
        for bit in range(32):
            words |= (rand(*words.shape) >= case["masked"]).int() << bit
        state["mask"] = words
    if case["op"] == "adjust_grad":
        state["g"] = torch.empty_like(x).normal_(0.0, 0.01, generator=g)
        state["g_shards"] = _shards(state["g"], W, 1)
    state["out"] = torch.empty_like(x)
    state["out_shards"] = _shards(state["out"], W, 1)
    return state


def _sizes(case):
    """The tensors' sizes: most of the elements in some, the others small, odd ones among them."""
    n, total = case["tensors"], case["elements"]
    rng = random.Random(n)
    w = [math.exp(rng.uniform(0.0, 6.0)) for _ in range(n)]
    sizes = [max(1, int(total * x / sum(w))) for x in w]
    sizes[0] = max(1, sizes[0] + total - sum(sizes))
    return sizes


def _types(case):
    return [("fp32" if i % 3 == 1 else "bf16") if case["dtype"] == "mixed" else case["dtype"] for i in range(case["tensors"])]


def _flat_places(case):
    """{type: (elements of its flat buffer, [(tensor, place)])}: each tensor on a 256-byte boundary, as frameworks lay them."""
    places = {}
    for i, (n, d) in enumerate(zip(_sizes(case), _types(case))):
        end, at = places.get(d, (0, []))
        at.append((i, end))
        step = 256 // BYTES[d]
        places[d] = (end + (n + step - 1) // step * step, at)
    return places


def _prepare_tensors(case, g):
    sizes = _sizes(case)
    sigma = case["norm"] / math.sqrt(sum(sizes))
    state = {"case": case, "grads": [None] * len(sizes), "outs": [None] * len(sizes), "flat": {}, "flat_out": {},
             "norm": torch.empty(1, device="cuda")}
    for d, (n, at) in _flat_places(case).items():
        flat = torch.zeros(n, dtype=DTYPES[d], device="cuda")
        state["flat"][d] = flat
        out = torch.zeros_like(flat) if case["op"] == "clip" else None
        state["flat_out"][d] = out
        for i, lo in at:
            state["grads"][i] = flat[lo:lo + sizes[i]].normal_(0.0, sigma, generator=g)
            state["outs"][i] = None if out is None else out[lo:lo + sizes[i]]
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

MAX_NORM = 1.0


def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    return {"embed": _plain_embed, "embed_grad": _plain_embed_grad, "adjust": _plain_adjust,
            "adjust_grad": _plain_adjust_grad, "norm": _plain_norm, "clip": _plain_clip}[case["op"]](state, case)


ADJUST = ("history", "n_history", "n_prompt", "repetition", "frequency", "presence", "bias_ids", "bias", "mask")


def _run_own(state, case):
    import collective_reduction_math_gb300 as mr
    op = case["op"]
    if op == "embed":
        mr.mr_embedding(state["shards"], state["ids"], state["out"], scale=case["scale"])
        return {"out": state["out"]}
    if op == "embed_grad":
        mr.mr_embedding_grad(state["g"], state["ids"], state["shards"], scale=case["scale"], accumulate=case["accumulate"])
        return {"grad": state["table"]}
    if op == "adjust":
        mr.mr_adjust_logits(state["logits"], state["out_shards"], **{n: state[n] for n in ADJUST})
        return {"out": state["out"]}
    if op == "adjust_grad":
        mr.mr_adjust_logits_grad(state["logits"], state["g_shards"], state["out_shards"],
                                 **{n: state[n] for n in ADJUST if not n.startswith("bias")})
        return {"grad": state["out"]}
    if op == "norm":
        mr.mr_grad_norm(state["grads"], state["norm"])
        return {"norm": state["norm"]}
    mr.mr_clip_grad_norm(state["grads"], state["outs"], MAX_NORM, norm=state["norm"])
    return {"norm": state["norm"], "out": state["flat_out"]}


# ---- the plain forms ----

def _plain_embed(state, case):
    ids = state["ids"]
    out = state["table"][ids.clamp(min=0)].float() * case["scale"]
    out.masked_fill_((ids < 0)[:, None], 0.0)
    return {"out": out.to(state["out"].dtype)}


def _plain_embed_grad(state, case):
    ids, table = state["ids"], state["table"]
    g = state["g"].float() * case["scale"]
    g.masked_fill_((ids < 0)[:, None], 0.0)
    # in 32 bits; a bf16 table is rounded once, at the end
    if case["accumulate"]:
        total = table if table.dtype == torch.float32 else table.float()
    else:
        total = torch.zeros(table.shape, device=table.device)
    total.index_add_(0, ids.clamp(min=0), g)
    if total is not table:
        table.copy_(total)
    return {"grad": table}


def _counts(state, case):
    """Occurrences of each column: among a row's whole history, and among what it said itself."""
    ids = state["history"]
    at = torch.arange(ids.shape[1], device=ids.device)[None, :]
    there = (at < state["n_history"][:, None]) & (ids >= 0)
    said = there & (at >= state["n_prompt"][:, None])
    none = torch.zeros(state["x"].shape, device=ids.device)
    ids = ids.clamp(min=0)
    return none.scatter_add(1, ids, there.float()), none.scatter_add(1, ids, said.float())


def _allowed(state, case):
    col = torch.arange(case["vocab"], dtype=torch.int32, device="cuda")
    return (state["mask"][:, (col // 32).long()] >> (col % 32)[None, :]) & 1


def _plain_adjust(state, case):
    y = state["x"].to(torch.float32, copy=True)
    if case["history"]:
        seen, said = _counts(state, case)
        rep = state["repetition"][:, None]
        y = torch.where(seen > 0, torch.where(y > 0, y / rep, y * rep), y)
        y -= state["frequency"][:, None] * said
        y -= state["presence"][:, None] * (said > 0)
    if case["bias"]:
        y.scatter_add_(1, state["bias_ids"], state["bias"])
    if case["masked"]:
        y.masked_fill_(_allowed(state, case) == 0, -math.inf)
    return {"out": y.to(state["x"].dtype)}


def _plain_adjust_grad(state, case):
    g = state["g"].to(torch.float32, copy=True)
    if case["history"]:
        seen, _ = _counts(state, case)
        rep = state["repetition"][:, None]
        g = torch.where(seen > 0, torch.where(state["x"] > 0, g / rep, g * rep), g)
    if case["masked"]:
        g.masked_fill_(_allowed(state, case) == 0, 0.0)
    return {"grad": g.to(state["x"].dtype)}


def _norm64(state):
    return torch.stack([f.float().square().sum(dtype=torch.float64) for f in state["flat"].values()]).sum().sqrt()


def _plain_norm(state, case):
    return {"norm": _norm64(state).float()[None]}


def _plain_clip(state, case):
    norm = _norm64(state)
    coef = (MAX_NORM / norm).clamp(max=1.0).float()
    return {"norm": norm.float()[None], "out": {d: (f.float() * coef).to(f.dtype) for d, f in state["flat"].items()}}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _distinct(case):
    """Distinct tokens of a batch, on average."""
    return float((-np.expm1((case["rows"] - _left_out(case)) * np.log1p(-_token_weights(case["vocab"])))).sum())


def work(case):
    op = case["op"]
    if op in ("norm", "clip"):
        sizes, types = _sizes(case), _types(case)
        b = sum(n * BYTES[d] for n, d in zip(sizes, types))
        return {"bytes": b * (2 if op == "clip" else 1), "flops": (3.0 if op == "clip" else 2.0) * sum(sizes)}
    T, V = case["rows"], case["vocab"]
    b = BYTES[case["dtype"]]
    if op in ("embed", "embed_grad"):
        H, on, rows = case["hidden"], T - _left_out(case), _distinct(case)
        if op == "embed":
            return {"bytes": 8 * T + (rows + T) * H * b, "flops": float(on * H)}
        table = BYTES[case["table"]] * H * (2 * rows if case["accumulate"] else V)
        return {"bytes": 8 * T + on * H * b + table, "flops": 1.0 * on * H + rows * H}
    # the history in its mean length; a gradient reads the scores of the tokens there alone
    said = 0.75 * case["history"]
    small = T * (8 * said + 12 * case["bias"] + (V / 8 if case["masked"] else 0) + (28 if said else 0))
    return {"bytes": 2 * T * V * b + small + (T * said * b if op == "adjust_grad" else 0), "flops": 1.0 * T * V}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    state = prepare(case, seed)
    return {"embed": _exact_embed, "embed_grad": _exact_embed_grad, "adjust": _exact_adjust, "adjust_grad": _exact_adjust,
            "norm": _exact_tensors, "clip": _exact_tensors}[case["op"]](case, state)


def _exact_embed(case, st):
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    on = (st["ids"] >= 0).nonzero()[:, 0]
    out[on] = st["table"].index_select(0, st["ids"][on]).double() * case["scale"]
    return {"out": out}


def _exact_embed_grad(case, st):
    on = (st["ids"] >= 0).nonzero()[:, 0]
    order = st["ids"][on].sort(stable=True)
    ids, n = order.values.unique_consecutive(return_counts=True)
    out = st["table"].double() if case["accumulate"] else torch.zeros(st["table"].shape, dtype=torch.float64, device="cuda")
    step = 512      # columns at a time
    last = n.cumsum(0) - 1
    for c in range(0, case["hidden"], step):
        sums = st["g"][:, c:c + step][on[order.indices]].double().cumsum(0)[last]
        sums[1:] -= sums[:-1].clone()
        out[ids, c:c + step] += sums * case["scale"]
    return {"grad": out}


def _exact_adjust(case, st):
    T, V = case["rows"], case["vocab"]
    grad = case["op"] == "adjust_grad"
    parts, step = [], max(1, (1 << 26) // V)
    for lo in range(0, T, step):
        hi = min(T, lo + step)
        x = st["x"][lo:hi].double()
        y = st["g"][lo:hi].double() if grad else x.clone()
        row = torch.arange(hi - lo, device="cuda")[:, None]
        if case["history"]:
            at = torch.arange(case["history"], device="cuda")
            flat = row * V + st["history"][lo:hi]
            here = at < st["n_history"][lo:hi, None]
            later = here & (at >= st["n_prompt"][lo:hi, None])
            all_of = torch.bincount(flat[here], minlength=x.numel()).view(x.shape)
            own_of = torch.bincount(flat[later], minlength=x.numel()).view(x.shape).double()
            factor = st["repetition"][lo:hi, None].double().expand(x.shape).clone()
            up = x > 0
            factor[up] = 1.0 / factor[up]
            factor[all_of == 0] = 1.0
            y *= factor
            if not grad:
                y -= st["frequency"][lo:hi, None].double() * own_of + st["presence"][lo:hi, None].double() * own_of.clamp(max=1.0)
        if case["bias"] and not grad:
            y[row.expand(-1, case["bias"]), st["bias_ids"][lo:hi]] += st["bias"][lo:hi].double()
        if case["masked"]:
            words = st["mask"][lo:hi].long() & 0xFFFFFFFF
            bits = torch.stack([(words >> b) & 1 for b in range(32)], 2).view(hi - lo, -1)[:, :V]
            y = torch.where(bits == 1, y, torch.full_like(y, 0.0 if grad else -math.inf))
        parts.append(y)
    return {"grad" if grad else "out": torch.cat(parts)}


def _exact_tensors(case, st):
    total = sum(float(torch.dot(p.double(), p.double())) for t in st["grads"] for p in t.split(1 << 26))
    norm = math.sqrt(total)
    out = {"norm": torch.tensor([norm], dtype=torch.float64)}
    if case["op"] == "clip":
        out["out"] = {d: f.double() * min(1.0, MAX_NORM / norm) for d, f in st["flat"].items()}
    return out
