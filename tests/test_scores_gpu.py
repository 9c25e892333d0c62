"""The token-score kernels against their 64-bit definitions, at the sizes,
layouts and values where they can go wrong.

Tolerances, from the arithmetic (u = 2^-24, half an fp32 step):
  - an exponential of t = y - m: the 2^x instruction is off by 2^-22
    relative, its argument by two roundings of |t|, so |t| 2^-22 more.  Terms
    with |t| > 32 are below 2^-46 of the largest.  A sum of such terms is off
    by at most 2^-22 + 32 * 2^-22 relative, and by its rounding: at most 64
    additions deep here, 64 u.  Together below 2^-16: REL.
  - log probabilities, logs of sums: REL absolute, plus u per unit of the
    result's own size and of t.
  - gradients: REL relative to the probability they are made of, then the
    rounding to the type: half a step, 2^-8 (bf16) or 2^-24 (fp32).
"""
import numpy as np
import pytest

import score_ref as ref

pytestmark = pytest.mark.gpu
REL = 2.0 ** -16
U = 2.0 ** -24
HALF_STEP = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8}
TINY = {"fp32": 2.0 ** -126, "bf16": 2.0 ** -126}     # the 2^x instruction flushes below it


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


def _dt(dtype):
    import torch
    return {"fp32": torch.float32, "bf16": torch.bfloat16}[dtype]


def _scores(seed, T, V, dtype, masked=0.0):
    """[T, V] scores on the CPU, exact in the type."""
    import torch
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, V, generator=g) * 2.5
    hot = torch.randint(0, V, (T, 4), generator=g)
    x.scatter_(1, hot, torch.rand(T, 4, generator=g) * 8 + 2)
    if masked:
        x.masked_fill_(torch.rand(T, V, generator=g) < masked, float("-inf"))
        x[:, 0] = 0.5
    return x.to(_dt(dtype))


class Rows:
    """W rank buffers of [T, V] scores inside fenced allocations: `pad` columns
    between rows, `offset` elements before the first."""

    FENCE = 64

    def __init__(self, W, T, V, dtype, pad=0, offset=0, fill=None):
        import torch
        self.cuts = [r * V // W for r in range(W + 1)]
        self.raw, self.views = [], []
        for r in range(W):
            w = self.cuts[r + 1] - self.cuts[r]
            n = T * (w + pad) + offset + 2 * self.FENCE
            raw = torch.full((n,), 77.0, dtype=_dt(dtype), device="cuda")
            v = torch.as_strided(raw, (T, w), (w + pad, 1), self.FENCE + offset)
            if fill is not None:
                v.copy_(fill[:, self.cuts[r]:self.cuts[r + 1]])
            self.raw.append(raw)
            self.views.append(v)

    def fenced(self):
        """Nothing outside the views was written."""
        for raw, v in zip(self.raw, self.views):
            keep = raw.clone()
            keep_v = keep.as_strided(v.shape, v.stride(), v.storage_offset())
            keep_v.fill_(77.0)
            assert bool((keep == 77.0).all()), "written outside the rows"

    def host(self):
        import torch
        return torch.cat([v.float().cpu() for v in self.views], 1).double().numpy()


def _close(got, want, tol, what=""):
    got, want, tol = np.asarray(got, np.float64), np.asarray(want, np.float64), np.broadcast_to(tol, np.shape(want))
    assert got.shape == want.shape, what
    odd = ~np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    assert np.array_equal(got[odd & ~np.isnan(want)], want[odd & ~np.isnan(want)]), f"{what}: infinities differ"
    err = np.abs(got[~odd] - want[~odd])
    over = err > tol[~odd]
    assert not over.any(), f"{what}: {over.sum()} of {err.size} off, worst {err[over].max()} (want {want[~odd][over][0]})"


def _forward(mr, rows, ids, scale, k, stream=None):
    import torch
    T = rows.views[0].shape[0]
    o = {n: torch.full((T,) + s, 77.0, device="cuda") for n, s in (("lp", ()), ("h", ()), ("stats", (2,)), ("top_lp", (max(k, 1),)))}
    o["top"] = torch.full((T, max(k, 1)), 77, dtype=torch.int64, device="cuda")
    mr.mr_logprob(rows.views, None if ids is None else torch.as_tensor(ids).cuda(), scale=scale, logprob=None if ids is None else o["lp"],
                  entropy=o["h"], stats=o["stats"], top_ids=o["top"] if k else None, top_logprob=o["top_lp"] if k else None,
                  stream=stream)
    torch.cuda.synchronize()
    return o


def _check_forward(x, ids, scale, k, o, what):
    T = x.shape[0]
    for t in range(T):
        lp, h, stats, top, top_lp = ref.logprob_row(x[t], None if ids is None else int(ids[t]), scale, k)
        top_lp = [v if v >= -3.4028235e38 or v != v else -np.inf for v in top_lp]      # below fp32's range
        spread = abs(stats[1]) + 1 if np.isfinite(stats[1]) else 1.0
        w = f"{what} row {t}"
        if ids is not None:
            _close(o["lp"][t].item(), lp, REL + (4 * U * (abs(lp) + spread) if np.isfinite(lp) else 0), w + " logprob")
        # u/s and log s each off by REL of terms no larger than the entropy and the spread
        _close(o["h"][t].item(), h, 2 * REL * (spread + (h if np.isfinite(h) else 0)), w + " entropy")
        _close(o["stats"][t, 0].item(), np.float64(np.float32(stats[0])), U * (abs(stats[0]) if np.isfinite(stats[0]) else 0), w + " max")
        _close(o["stats"][t, 1].item(), stats[1], REL + U * spread, w + " log sum")
        if k:
            assert o["top"][t, :k].tolist() == list(top), w + " top ids"
            fin = np.array([abs(v) if np.isfinite(v) else 0 for v in top_lp])
            _close(o["top_lp"][t, :k].cpu().numpy(), top_lp, REL + 4 * U * (fin + spread), w + " top logprob")


# (W, T, V, scale, k, pad, offset): one column, fewer columns than ranks, both
# sides of a vector, a run and a superblock, rows off every boundary, many rows
SHAPES = [(1, 1, 1, 1.0, 1, 0, 0), (2, 3, 2, 1.0, 2, 0, 0), (8, 3, 5, 0.7, 5, 3, 1), (64, 2, 63, 1.0, 20, 1, 0),
          (1, 5, 7, 2.0, 7, 0, 0), (1, 4, 255, 1.0, 64, 0, 0), (1, 4, 256, 1.0, 3, 0, 0), (1, 4, 257, 1.0, 64, 0, 3),
          (3, 4, 1000, 1.25, 20, 0, 0), (1, 3, 1023, 1.0, 1, 1, 0), (1, 3, 1024, 1.0, 64, 0, 0), (1, 3, 1025, 1.0, 5, 0, 0),
          (1, 3, 513, 1.0, 5, 0, 2), (8, 5, 8192, 0.5, 20, 8, 0), (64, 2, 20011, 1.0, 33, 0, 0), (1, 1, 50001, 1.0, 20, 0, 0),
          (5, 7, 16384, 1.0, 0, 5, 5), (2, 700, 1537, 1.0, 4, 0, 0), (1, 1100, 300, 1.0, 2, 0, 0), (1, 2, 131072, 1.0, 64, 0, 0)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("W,T,V,scale,k,pad,offset", SHAPES)
def test_logprob(mr, dtype, W, T, V, scale, k, pad, offset):
    x = _scores(W * 1000 + V, T, V, dtype)
    rng = np.random.default_rng(V)
    ids = rng.integers(0, V, T)
    if T > 2:
        ids[1], ids[2] = -100, 0
    if T > 4:
        ids[3], ids[4] = V - 1, V + 5
    rows = Rows(W, T, V, dtype, pad, offset, x)
    o = _forward(mr, rows, ids, scale, k)
    xs = x.double().numpy()
    step = max(1, T // 40)
    sel = sorted(set(range(0, T, step)) | set(range(min(T, 6))) | {T - 1})
    _check_forward(xs[sel], ids[sel], float(np.float32(scale)), k, {n: v[sel] for n, v in o.items()}, f"{dtype} {W}x{V}")
    rows.fenced()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("W,V", [(1, 600), (3, 2500), (8, 40)])
def test_logprob_odd_values(mr, dtype, W, V):
    """Masks, the lowest values, ties, signed zeros, infinities and NaN."""
    import torch
    ninf = float("-inf")
    x = _scores(5, 16, V, dtype).float()
    lowest = torch.finfo(_dt(dtype)).min
    x[0] = ninf                                         # nothing left
    x[1] = ninf
    x[1, V - 1] = -3.0                                  # one place left
    x[2] = lowest                                       # the lowest value everywhere
    x[3] = lowest
    x[3, V // 2] = 1.0
    x[4] = ninf
    x[4, V // 3:] = lowest                              # masked by both
    x[5] = 1.5                                          # ties everywhere
    x[6] = 0.0
    x[6, ::2] = -0.0                                    # equal zeros
    x[7, V // 2] = float("nan")
    x[8, 3] = float("inf")
    x[9] = ninf
    x[9, 5] = float("nan")
    x[10, ::2] = ninf
    x[11] = torch.linspace(-80, 80, V)                  # a steep row
    x[12] = -1e30
    x[12, 7] = 20.0
    x[13, :] = 3e4
    x[14] = torch.where(torch.arange(V) % 3 == 0, 2.0, 1.0)
    ids = np.array([0, V - 1, 1, V // 2, V - 1, 4, 1, 2, 3, 5, 0, V - 1, 7, 1, 3, 2])
    x = x.to(_dt(dtype))
    rows = Rows(W, 16, V, dtype, 1, 0, x)
    for k in (0, 1, 20, min(64, V)):
        o = _forward(mr, rows, ids, 1.0, k)
        _check_forward(x.double().numpy(), ids, 1.0, k, o, f"{dtype} k={k}")
    o = _forward(mr, rows, None, 1.0, 4)                # no token asked for
    _check_forward(x.double().numpy(), None, 1.0, 4, o, dtype)


@pytest.mark.parametrize("order", ["up", "down", "blocks", "last run"])
def test_top_k_where_it_lies(mr, order):
    """The best scores bunched in one run, in order, or one a run."""
    import torch
    V = 20000
    x = torch.zeros(2, V)
    if order == "up":
        x[:] = torch.arange(V) * 1e-3
    elif order == "down":
        x[:] = -torch.arange(V) * 1e-3
    elif order == "blocks":
        x[:, ::128] = 5.0
        x[0, 128 * 77] = 6.0
    else:
        x[:, -64:] = torch.arange(64) * 0.25 + 1
    for dtype in ("fp32", "bf16"):
        xs = x.to(_dt(dtype))
        rows = Rows(1, 2, V, dtype, 0, 0, xs)
        o = _forward(mr, rows, np.array([0, V - 1]), 1.0, 64)
        for t in range(2):
            assert o["top"][t].tolist() == ref.logprob_row(xs[t].double().numpy(), 0, 1.0, 64)[3], (order, dtype)


@pytest.mark.parametrize("T", [3, 1000])        # one row a cluster, and several
@pytest.mark.parametrize("k", [1, 20, 64])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_top_k_ties_and_masks(mr, dtype, k, T):
    """Few places left by a mask, equal scores in floods, scores crowded in a run."""
    V = 9001
    x = _scores(61, T, V, dtype).float()
    x[0] = float("-inf")
    x[0, [5, 4000, 9000]] = 1.0
    x[1] = 2.0
    x[2] = (x[2] * 2).round() / 2
    if T > 3:
        x[-1, :300] += 50.0
        x[-2] = float("-inf")
        x[-3, 100:] = float("-inf")
        x[-4] = 0.0
        x[-4, ::7] = 1.0
    x = x.to(_dt(dtype))
    rows = Rows(2, T, V, dtype, 0, 0, x)
    o = _forward(mr, rows, np.zeros(T, np.int64), 1.0, k)
    for t in {0, 1, 2, T - 1, T - 2, T - 3, T - 4} & set(range(T)):
        want = ref.logprob_row(x[t].double().numpy(), 0, 1.0, k)
        assert o["top"][t].tolist() == want[3], t
        _close(o["top_lp"][t].cpu().numpy(), want[4], REL + 4 * U * 128, f"row {t}")


@pytest.mark.parametrize("T", [7, 700])         # a row on many CTAs, and rows in turn on few
@pytest.mark.parametrize("k", [20, 64])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_top_k_of_long_candidate_lists(mr, dtype, k, T):
    """More scores at or above the bound than are ranked at a time, in a long row."""
    V = 70001
    x = _scores(67, 7, V, dtype).float()
    x[0] = 0.0
    x[1, 1000:1100] = x[2, :100]
    x[1, :1000] = x[1, 1100:] = float("-inf")
    x[2, 5000:5256] += 50.0
    x[3, 30000:32000] += 50.0
    x[4, ::23] = float("nan")
    x[5] = x[5].sort()[0]
    x[6] = (x[6] * 2).round() / 2
    x = x.to(_dt(dtype))
    rows = Rows(2, T, V, dtype, 0, 0, x.repeat((T + 6) // 7, 1)[:T].contiguous())
    o = _forward(mr, rows, np.zeros(T, np.int64), 1.0, k)
    for t in range(7):
        want = ref.logprob_row(x[t].double().numpy(), 0, 1.0, k)
        for u in (t, T - 7 + t):
            assert o["top"][u].tolist() == want[3], u
            _close(o["top_lp"][u].cpu().numpy(), want[4], REL + 4 * U * 128, f"row {u}")


@pytest.mark.parametrize("scale", [0.7, 3.0])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_lowest_values_at_a_scale(mr, dtype, scale):
    """Rows of the type's lowest value, whose scaled scores round by whole
    units or overflow to -inf."""
    import torch
    V, T = 1500, 4
    low = torch.finfo(_dt(dtype)).min
    x = _scores(71, T, V, dtype).float()
    x[0] = low
    x[1] = low
    x[1, 77] = 1.0
    x[2, ::2] = low
    x = x.to(_dt(dtype))
    rows, out = Rows(2, T, V, dtype, 0, 0, x), Rows(2, T, V, dtype)
    ids = np.array([3, 77, 1, 2])
    o = _forward(mr, rows, ids, scale, 3)
    sc = float(np.float32(scale))
    y_low = float(np.float32(np.float64(x[0, 0].item()) * sc)) if abs(x[0, 0].item()) * sc < 3.4028235e38 else -np.inf
    if y_low == -np.inf:        # a masked row in fp32
        assert o["stats"][0].tolist() == [-np.inf, 0.0] and o["lp"][0].item() == -np.inf and o["h"][0].item() == 0
    else:
        _close(o["stats"][0].cpu().numpy(), [y_low, np.log(V)], [0.0, REL])
        _close(o["lp"][0].item(), -np.log(V), REL)
        _close(o["h"][0].item(), np.log(V), 2 * REL * 8)
    assert o["top"][0].tolist() == [0, 1, 2]
    _check_forward(x[1:].double().numpy(), ids[1:], sc, 3, {n: v[1:] for n, v in o.items()}, "lowest")
    g = torch.ones(T, device="cuda")
    mr.mr_logprob_grad(rows.views, torch.from_numpy(ids).cuda(), o["stats"], out.views, g_logprob=g, scale=scale)
    torch.cuda.synchronize()
    got = out.host()
    if y_low == -np.inf:
        want = np.zeros(V)
        want[3] = 0.0 if got[0, 3] == 0 else sc      # the place itself is finite: either reading is a number
    else:
        want = np.full(V, -sc / V)
        want[3] += sc
    _close(got[0], want, HALF_STEP[dtype] * np.abs(want) + 2 * REL * sc / V + 4 * U * (np.arange(V) == 3))
    for t in (1, 2, 3):
        w = ref.logprob_grad_row(x[t].double().numpy(), int(ids[t]), sc, 1.0, 0.0)
        _close(got[t], w, _prob_tol(w, np.abs(w) + 4 * U / REL * sc * (np.arange(V) == ids[t]), dtype))


def _stats(x, scale, ids=None):
    out = []
    for t in range(x.shape[0]):
        y = x[t] * scale
        s = ref.lse_parts(y)
        if ids is not None:
            rest = y.copy()
            rest[ids[t][(ids[t] >= 0) & (ids[t] < y.size)]] = -np.inf
            s = s + ref.lse_parts(rest)
        out.append(s)
    return np.array(out, np.float32)


GRAD_SHAPES = [(1, 1, 1, 1.0, 0, 0, 0), (8, 3, 5, 0.7, 3, 1, 1), (64, 2, 63, 1.0, 1, 0, 0), (1, 4, 257, 1.0, 0, 3, 0),
               (3, 4, 1000, 1.25, 0, 0, 0), (1, 3, 1023, 1.0, 1, 0, 0), (1, 3, 1025, 1.0, 0, 0, 5), (8, 5, 8192, 0.5, 8, 0, 0),
               (5, 7, 16384, 1.0, 5, 5, 5), (2, 300, 1537, 1.0, 0, 0, 0), (1, 2, 131072, 1.0, 0, 0, 0)]


def _prob_tol(grad, parts, dtype):
    """REL of the probabilities a gradient is made of, then one rounding."""
    return 2 * REL * parts + HALF_STEP[dtype] * (np.abs(grad) + 2 * REL * parts) + TINY[dtype]


@pytest.mark.parametrize("ent,lp", [(False, True), (True, True), (True, False)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("W,T,V,scale,pad,offset,out_offset", GRAD_SHAPES)
def test_logprob_grad(mr, dtype, W, T, V, scale, pad, offset, out_offset, ent, lp):
    import torch
    x = _scores(V + 1, T, V, dtype, masked=0.3 if V > 5 else 0.0)
    rng = np.random.default_rng(V)
    ids = rng.integers(0, V, T)
    if T > 2:
        ids[1], ids[2] = -1, V
    xs, scale = x.double().numpy(), float(np.float32(scale))
    stats = _stats(xs, scale)
    h = np.array([ref.logprob_row(r, None, scale, 0)[1] for r in xs], np.float32)
    g_lp, g_h = rng.normal(0, 1, T).astype(np.float32), rng.normal(0, 1, T).astype(np.float32)
    up = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    want = np.stack([ref.logprob_grad_row(xs[t], int(ids[t]) if lp else None, scale, g_lp[t] if lp else 0.0, g_h[t] if ent else 0.0)
                     for t in range(T)])
    p = np.exp(np.stack([ref.log_softmax(r * scale) for r in xs]))
    logp = np.where(p > 0, np.log(np.maximum(p, 1e-300)), 0.0)
    parts = scale * ((np.abs(g_lp)[:, None] * p if lp else 0) + (np.abs(g_h)[:, None] * p * (np.abs(logp) + h[:, None] + 1) if ent else 0))
    if lp:
        on = (ids >= 0) & (ids < V)
        parts[np.nonzero(on)[0], ids[on]] += scale * np.abs(g_lp[on]) * 4 * U / REL
    for in_place in (False, True):
        rows = Rows(W, T, V, dtype, pad, offset, x)
        out = rows if in_place else Rows(W, T, V, dtype, pad, offset + out_offset)
        mr.mr_logprob_grad(rows.views, up(ids) if lp else None, up(stats), out.views, g_logprob=up(g_lp) if lp else None,
                           entropy=up(h) if ent else None, g_entropy=up(g_h) if ent else None, scale=scale)
        torch.cuda.synchronize()
        _close(out.host(), want, _prob_tol(want, parts, dtype), f"{dtype} in place {in_place}")
        out.fenced()


def _teacher(rng, T, V, K, tail, holes):
    ids = np.stack([rng.permutation(V)[:K] if V < 5000 else rng.choice(V, K, replace=False) for _ in range(T)]).astype(np.int64)
    if tail:
        val = np.log(rng.dirichlet(np.ones(K), T) * rng.uniform(0.3, 0.99, (T, 1)) + 1e-12)
    else:
        val = rng.normal(0, 2, (T, K))
    if holes and T > 2:
        ids[0, : K // 2] = -1
        ids[1] = -5
        val[2, -1] = -np.inf
    return ids, val.astype(np.float32)


# (W, T, V, K, scale, pad, offset, out_offset)
DISTILL_SHAPES = [(1, 1, 2, 1, 1.0, 0, 0, 0), (1, 3, 5, 5, 1.0, 0, 0, 0), (8, 4, 6, 3, 0.7, 3, 1, 1), (64, 3, 63, 20, 1.0, 1, 0, 0),
                  (1, 4, 257, 100, 1.0, 0, 3, 0), (3, 4, 1000, 33, 1.25, 0, 0, 0), (1, 3, 1025, 128, 1.0, 0, 0, 5),
                  (8, 5, 8192, 64, 0.5, 8, 0, 0), (5, 7, 16384, 31, 1.0, 5, 5, 5), (2, 400, 1537, 8, 1.0, 0, 0, 0),
                  (1, 2, 131072, 128, 1.0, 0, 0, 0)]


def _run_distill(mr, which, rows, out, ids, val, g, stats, **kw):
    import torch
    T = rows.views[0].shape[0]
    up = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    loss = torch.full((T,), 77.0, device="cuda")
    st = torch.full((T, 4), 77.0, device="cuda")
    if which == "forward":
        mr.mr_distill_topk(rows.views, up(ids), up(val), loss, stats=st, **kw)
    elif which == "grad":
        mr.mr_distill_topk_grad(rows.views, up(ids), up(val), up(stats), up(g), out.views, **kw)
    else:
        mr.mr_distill_topk_step(rows.views, up(ids), up(val), up(g), loss, out.views, **kw)
    torch.cuda.synchronize()
    return loss.cpu().numpy(), st.cpu().numpy()


def _check_distill(mr, dtype, W, x, ids, val, scale, tail, t_scale, pad, offset, out_offset):
    T, V = x.shape
    xs, scale = x.double().numpy(), float(np.float32(scale))
    g = np.random.default_rng(9).normal(0, 1, T).astype(np.float32)
    res = [ref.distill_row(xs[t], ids[t], val[t].astype(np.float64), scale, tail, t_scale, float(g[t])) for t in range(T)]
    loss, stats, grad = np.array([r[0] for r in res]), np.array([r[1] for r in res]), np.stack([r[2] for r in res])
    size = np.array([r[3] for r in res])
    kw = dict(mode="tail" if tail else "renorm", scale=scale, teacher_scale=t_scale)
    # q is off by REL/8 (exact exponentials), the remainder by a few u of 1, log p by REL and 4 u of itself
    with np.errstate(divide="ignore", invalid="ignore"):
        q_rest = np.array([max(2.0 ** -20, 1 - np.exp(v[i >= 0].astype(np.float64)).sum()) if tail else 1.0 for v, i in zip(val, ids)])
        spread = np.where(np.isfinite(stats[:, 1]), np.abs(stats[:, 0]) + np.abs(stats[:, 2]), 0)
    spread = np.where(np.isfinite(spread), spread, 0)
    loss_tol = 2 * REL * size + 64 * U * (size + spread) + (64 * U * (1 + np.abs(np.log(q_rest))) if tail else 0)
    p = np.exp(np.stack([ref.log_softmax(r * scale) for r in xs]))
    rest = xs * scale
    parts = np.where(np.isnan(p), 0, p)
    for t in range(T):
        i = ids[t][(ids[t] >= 0) & (ids[t] < V)]
        rest[t, i] = -np.inf
        r = np.exp(ref.log_softmax(rest[t]))
        if tail:
            # the remaining mass is off by a few u of 1: that much of softmax over the outside
            parts[t] += np.where(np.isnan(r), 0, r) * (q_rest[t] if q_rest[t] > 2.0 ** -20 else 1.0)
            parts[t] += np.where(np.isnan(r), 0, r) * 64 * U / REL
        q = np.exp(val[t][ids[t] >= 0].astype(np.float64)) if tail else np.ones(int((ids[t] >= 0).sum()))
        j = ids[t][ids[t] >= 0]
        parts[t, j[j < V]] += np.where(np.isfinite(q), q, 0)[j < V]
    parts *= scale * np.abs(g)[:, None]
    rows = Rows(W, T, V, dtype, pad, offset, x)
    got, st = _run_distill(mr, "forward", rows, None, ids, val, g, None, **kw)
    _close(got, loss, loss_tol, "loss")
    _close(st[:, 0::2], stats[:, 0::2].astype(np.float32).astype(np.float64),
           U * np.where(np.isfinite(stats[:, 0::2]), np.abs(stats[:, 0::2]), 0), "maxima")
    _close(st[:, 1::2], stats[:, 1::2], REL + U * np.where(np.isfinite(stats[:, 1::2]), np.abs(stats[:, 1::2]), 0), "log sums")
    for which in ("grad", "step"):
        for in_place in (False, True):
            rows = Rows(W, T, V, dtype, pad, offset, x)
            out = rows if in_place else Rows(W, T, V, dtype, pad, offset + out_offset)
            got, _ = _run_distill(mr, which, rows, out, ids, val, g, stats.astype(np.float32), **kw)
            if which == "step":
                _close(got, loss, loss_tol, "step loss")
            _close(out.host(), grad, _prob_tol(np.where(np.isnan(grad), 0, grad), parts, dtype), f"{which} in place {in_place}")
            out.fenced()


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("W,T,V,K,scale,pad,offset,out_offset", DISTILL_SHAPES)
def test_distill(mr, dtype, W, T, V, K, scale, pad, offset, out_offset, tail):
    x = _scores(V + 2, T, V, dtype)
    ids, val = _teacher(np.random.default_rng(V + K), T, V, K, tail, holes=V > 5)
    _check_distill(mr, dtype, W, x, ids, val, scale, tail, 1.0 if tail else 0.75, pad, offset, out_offset)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_distill_odd_values(mr, dtype, tail):
    """Rows with nothing left, masks inside and outside the list, a rest of
    vanishing mass, columns past the vocabulary, infinities and NaN."""
    import torch
    V, K, T, ninf = 2500, 4, 14, float("-inf")
    x = _scores(8, T, V, dtype).float()
    rng = np.random.default_rng(1)
    ids, val = _teacher(rng, T, V, K, tail, holes=False)
    x[0] = ninf                                         # nothing left: the loss is +inf
    x[1] = ninf
    x[1, torch.from_numpy(ids[1])] = 1.0                # only the list is left
    x[2, torch.from_numpy(ids[2])] = ninf               # the whole list is masked
    x[3, int(ids[3, 0])] = ninf
    x[4, ::2] = ninf
    x[4, torch.from_numpy(ids[4])] = 2.0
    x[5, torch.from_numpy(ids[5])] = 60.0               # a rest of vanishing mass
    x[6] = torch.finfo(_dt(dtype)).min
    x[7, 3] = float("nan")
    x[8, int(ids[8, 1])] = float("inf")
    ids[9, 2] = V + 3                                   # past the vocabulary
    val[10, :2] = -np.inf                               # no mass on two entries
    x[10, int(ids[10, 0])] = ninf                       # ... one of them masked: 0 log 0
    val[11, 0] = np.nan
    if not tail:
        val[12] = -np.inf                               # nothing to learn from
    ids[13, 1:] = -1
    if tail:
        val[13, 0] = 0.0                                # the whole mass on one entry
    _check_distill(mr, dtype, 3, x.to(_dt(dtype)), ids, val, 1.0, tail, 1.0, 1, 0, 0)


@pytest.mark.parametrize("dtype,V", [("bf16", 1_700_003), ("fp32", 900_001)])
def test_step_row_longer_than_shared_memory(mr, dtype, V):
    x = _scores(3, 2, V, dtype)
    ids, val = _teacher(np.random.default_rng(2), 2, V, 16, True, holes=False)
    _check_distill(mr, dtype, 1, x, ids, val, 1.0, True, 1.0, 0, 0, 0)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_gradients_against_differences(mr, dtype):
    """The GPU's gradient along a direction is the 64-bit loss's difference."""
    T, V, K = 3, 700, 6
    x = _scores(21, T, V, dtype)
    xs, rng = x.double().numpy(), np.random.default_rng(7)
    ids, val = _teacher(rng, T, V, K, True, holes=False)
    g = rng.normal(0, 1, T).astype(np.float32)
    rows, out = Rows(2, T, V, dtype, 0, 0, x), Rows(2, T, V, dtype)
    _run_distill(mr, "step", rows, out, ids, val, g, None, mode="tail")
    grad = out.host()
    for t in range(T):
        d = rng.normal(0, 1, V)
        f = lambda z: float(g[t]) * ref.distill_row(z, ids[t], val[t].astype(np.float64), 1.0, True, 1.0, 1.0)[0]  # noqa: B023,E731
        diff = (f(xs[t] + 1e-5 * d) - f(xs[t] - 1e-5 * d)) / 2e-5
        tol = 1e-6 + (HALF_STEP[dtype] + 4 * REL) * (np.abs(grad[t] * d).sum() + np.abs(g[t]) * 0.01)
        assert abs(diff - (grad[t] * d).sum()) < tol


def test_column_slices_of_one_buffer(mr):
    """Ranks that are column slices of one [T, V] buffer, in place too."""
    import torch
    T, V, W, K = 5, 3001, 3, 7
    x = _scores(31, T, V, "bf16")
    cut = [r * V // W for r in range(W + 1)]
    full = x.cuda()
    ids, val = _teacher(np.random.default_rng(3), T, V, K, False, holes=True)
    up = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    g = torch.ones(T, device="cuda")
    want = [torch.empty(T, cut[r + 1] - cut[r], dtype=torch.bfloat16, device="cuda") for r in range(W)]
    loss, loss2 = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    mr.mr_distill_topk_step([full[:, cut[r]:cut[r + 1]].contiguous() for r in range(W)], up(ids), up(val), g, loss, want)
    slices = [full[:, cut[r]:cut[r + 1]] for r in range(W)]
    mr.mr_distill_topk_step(slices, up(ids), up(val), g, loss2, slices)
    assert torch.allclose(loss, loss2, rtol=1e-5, atol=1e-5)
    a, b = torch.cat(want, 1).float(), full.float()
    assert torch.allclose(a, b, rtol=2 ** -7, atol=1e-6)


def test_repeats_streams_and_graphs(mr):
    """The same bits on every run, on a side stream and from a graph."""
    import torch
    T, V = 9, 33333
    rows = Rows(2, T, V, "bf16", 0, 0, _scores(41, T, V, "bf16"))
    ids = np.arange(T) * 7
    first = _forward(mr, rows, ids, 1.0, 20)
    again = _forward(mr, rows, ids, 1.0, 20)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = _forward(mr, rows, ids, 1.0, 20)
    o = {n: torch.zeros_like(v) for n, v in first.items()}
    dev_ids = torch.from_numpy(ids).cuda()
    out = Rows(2, T, V, "bf16")
    g_lp = torch.ones(T, device="cuda")

    def both():
        mr.mr_logprob(rows.views, dev_ids, logprob=o["lp"], entropy=o["h"], stats=o["stats"], top_ids=o["top"], top_logprob=o["top_lp"])
        mr.mr_logprob_grad(rows.views, dev_ids, o["stats"], out.views, g_logprob=g_lp)

    with torch.cuda.stream(s):
        both()
    s.synchronize()
    eager = out.host()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        both()
    for n in o:
        o[n].zero_()
    for v in out.views:
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for n in first:
        for other in (again, side, o):
            assert torch.equal(first[n], other[n]), n
    assert np.array_equal(out.host(), eager)


def test_far_rows(mr):
    """Rows whose offsets pass 2^32 elements."""
    import torch
    T, V, ld = 5, 5000, (1 << 30) + 8
    raw = torch.empty(4 * ld + V, dtype=torch.bfloat16, device="cuda")
    far = raw.as_strided((T, V), (ld, 1))
    x = _scores(51, T, V, "bf16")
    far.copy_(x)
    ids = np.array([0, 4999, 17, -1, 2500])
    near = Rows(1, T, V, "bf16", 0, 0, x)
    a = _forward(mr, near, ids, 1.0, 8)
    rows = Rows(1, 1, 1, "bf16")
    rows.views = [far]
    b = _forward(mr, rows, ids, 1.0, 8)
    for n in a:
        assert torch.equal(a[n], b[n]), n
    dev, out = torch.from_numpy(ids).cuda(), a["stats"]
    g = torch.ones(T, device="cuda")
    grad = Rows(1, T, V, "bf16")
    mr.mr_logprob_grad(near.views, dev, out, grad.views, g_logprob=g)
    mr.mr_logprob_grad([far], dev, out, [far], g_logprob=g)
    torch.cuda.synchronize()
    assert torch.equal(far.contiguous(), grad.views[0].contiguous())


def test_binding_refuses(mr):
    import torch
    x = [torch.zeros(4, 10, device="cuda"), torch.zeros(4, 11, device="cuda")]
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    lp = torch.zeros(4, device="cuda")
    mr.mr_logprob(x, ids, logprob=lp)
    for bad in ([x[1], x[0]], [x[0], x[1].t().contiguous().t()], [x[0], x[1].bfloat16()], [x[0], x[1][:3]], [x[0].flatten(), x[1]]):
        with pytest.raises(ValueError):
            mr.mr_logprob(bad, ids, logprob=lp)
    with pytest.raises(ValueError):
        mr.mr_logprob(x, ids.int(), logprob=lp)
    with pytest.raises(ValueError):
        mr.mr_logprob(x, ids, logprob=lp[:3])
    with pytest.raises(mr.MRError):
        mr.mr_logprob(x, ids)
    with pytest.raises(mr.MRError):
        mr.mr_logprob(x, ids, logprob=lp, scale=0.0)
    with pytest.raises(mr.MRError) as e:
        mr.mr_logprob_grad(x, ids, torch.zeros(4, 2, device="cuda"), [x[0][:, :10], x[0].new_zeros(4, 11)][::1], g_logprob=x[0].as_strided((4,), (1,)))
    assert e.value.status == 3
    torch.cuda.synchronize()
