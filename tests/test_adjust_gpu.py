"""Adjusted scores and their gradient against their definitions, at the sizes,
layouts, lists and masks where they can go wrong.  Bounds: step_ref's, plus half
a step of the type; columns that nothing concerns keep their bits."""
import numpy as np
import pytest

import step_ref as ref

pytestmark = pytest.mark.gpu
INF = float("inf")


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


class Shards:
    """W rank buffers of [T, V] inside fenced allocations: `pad` columns between rows, `offset` before the first."""

    FENCE = 64

    def __init__(self, W, x, pad=0, offset=0):
        import torch
        T, V = x.shape
        self.raw, self.views = [], []
        for r in range(W):
            lo, hi = r * V // W, (r + 1) * V // W
            raw = torch.full((T * (hi - lo + pad) + offset + 2 * self.FENCE,), 77.0, dtype=x.dtype, device="cuda")
            v = torch.as_strided(raw, (T, hi - lo), (hi - lo + pad, 1), self.FENCE + offset)
            v.copy_(x[:, lo:hi])
            self.raw.append(raw)
            self.views.append(v)

    def fenced(self):
        for raw, v in zip(self.raw, self.views):
            keep = raw.clone()
            keep.as_strided(v.shape, v.stride(), v.storage_offset()).fill_(77.0)
            assert bool((keep == 77.0).all()), "written outside the rows"

    def host(self):
        import torch
        return torch.cat([v.cpu() for v in self.views], 1)


def _lists(T, V, L, K, masked, seed, distinct_rows=True):
    """History with repeats, entries that are none, lengths from 0 to past the end; biases with repeats; a mask."""
    import torch
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.rand(*s, generator=g)  # noqa: E731
    a = {}
    if L:
        h = torch.randint(0, V, (T, L), generator=g)
        h[rand(T, L) < 0.3] = V - 1
        h[rand(T, L) < 0.1] = -1
        h[rand(T, L) < 0.05] = V + 5
        a["history"] = h
        a["n_history"] = torch.randint(0, L + 1, (T,), generator=g)
        a["n_prompt"] = (rand(T) * a["n_history"]).long()
        if T > 2:
            a["n_history"][0], a["n_history"][1], a["n_history"][2] = 0, L + 7, -3
            a["n_prompt"][1] = L + 9
        a["repetition"], a["frequency"], a["presence"] = 0.7 + rand(T), rand(T) * 0.6 - 0.1, rand(T) * 2 - 0.5
    if K:
        b = torch.randint(0, V, (T, K), generator=g)
        b[rand(T, K) < 0.1] = -1
        b[rand(T, K) < 0.05] = V
        a["bias_ids"], a["bias"] = b, torch.randn(T, K, generator=g) * 4
    if masked is not None:
        words = (V + 31) // 32
        bits = rand(T, words * 32) >= masked
        m = (bits.view(T, words, 32).long() << torch.arange(32)).sum(2)
        a["mask"] = torch.where(m >= 2 ** 31, m - 2 ** 32, m).int()
    return a


def _allowed(mask, t, V):
    if mask is None:
        return None
    words = mask[t].numpy().astype(np.int64) & 0xFFFFFFFF
    return ((words[:, None] >> np.arange(32)) & 1).astype(bool).ravel()[:V]


def _row_history(a, t):
    if "history" not in a:
        return np.zeros(0, np.int64), 0
    L = a["history"].shape[1]
    n = min(max(int(a["n_history"][t]), 0), L) if a.get("n_history") is not None else L
    p = min(max(int(a["n_prompt"][t]), 0), n) if a.get("n_prompt") is not None else 0
    return a["history"][t, :n].numpy(), p


def _value(a, name, t):
    return float(a[name][t]) if a.get(name) is not None else None


def _cuda(a):
    return {k: v.cuda() if v is not None else None for k, v in a.items()}


def _scores(T, V, dtype, seed):
    import torch
    x = torch.randn(T, V, generator=torch.Generator().manual_seed(seed)) * 3
    x[:, V // 2] = 0.0
    return x.to(_dt(dtype))


def _check(mr, x, dtype, W, a, pad=0, offset=0, in_place=False, what=""):
    import torch
    T, V = x.shape
    logits = Shards(W, x, pad, offset)
    out = logits if in_place else Shards(W, torch.full_like(x, 55.0), pad, offset)
    mr.mr_adjust_logits(logits.views, out.views, **_cuda(a))
    torch.cuda.synchronize()
    got = out.host()
    for t in range(T):
        h, p = _row_history(a, t)
        ids, b = (a["bias_ids"][t].numpy(), a["bias"][t].double().numpy()) if "bias" in a else ((), ())
        allowed = _allowed(a.get("mask"), t, V)
        row = x[t].double().numpy()
        want, bound = ref.adjusted_row(row, h, p, _value(a, "repetition", t), _value(a, "frequency", t), _value(a, "presence", t),
                                       ids, b, allowed)
        want = ref.in_type(want, dtype)     # the lowest value times a penalty
        still = (bound == 0) & np.isfinite(row) & ((want == row) if allowed is None else allowed & (want == row))
        ref.close(got[t].double().numpy(), want, bound * 1.01 + ref.rounded(want, dtype), f"{what} row {t}")
        assert np.array_equal(got[t].double().numpy()[still], row[still]), f"{what} row {t}: bits changed"
    out.fenced()
    if not in_place:
        assert torch.equal(logits.host().nan_to_num(9.0), x.nan_to_num(9.0))
        logits.fenced()


def _check_grad(mr, x, dtype, W, a, pad=0, offset=0, in_place=False, what=""):
    import torch
    T, V = x.shape
    a = {k: v for k, v in a.items() if not k.startswith("bias")}
    g = _scores(T, V, dtype, 77)
    logits, g_in = Shards(W, x, pad, offset), Shards(W, g, pad, offset)
    out = g_in if in_place else Shards(W, torch.full_like(g, 55.0), pad, offset)
    mr.mr_adjust_logits_grad(logits.views, g_in.views, out.views, **_cuda(a))
    torch.cuda.synchronize()
    got = out.host()
    for t in range(T):
        h, _ = _row_history(a, t)
        want, bound = ref.adjusted_grad_row(g[t].double().numpy(), x[t].double().numpy(), h, _value(a, "repetition", t),
                                            _allowed(a.get("mask"), t, V))
        want = ref.in_type(want, dtype)
        ref.close(got[t].double().numpy(), want, np.where(bound > 0, bound + ref.rounded(want, dtype), 0.0), f"{what} row {t}")
    out.fenced()


# (W, T, V, L, K, masked, pad, offset): one column, fewer columns than ranks, vectors, words and
# windows with something on both sides, rows off every boundary
SHAPES = [(1, 1, 1, 1, 1, 0.5, 0, 0), (8, 3, 5, 4, 2, 0.3, 3, 1), (64, 4, 63, 9, 3, 0.5, 1, 0), (1, 5, 31, 40, 0, 0.5, 0, 0),
          (1, 5, 33, 0, 7, 0.9, 0, 0), (2, 4, 257, 300, 5, None, 5, 3), (3, 4, 1000, 20, 20, 0.2, 0, 0), (1, 3, 8191, 64, 9, 0.99, 0, 0),
          (1, 3, 8192, 200, 0, 0.5, 0, 0), (1, 3, 8193, 200, 30, 1.0, 0, 0), (5, 4, 20011, 999, 64, 0.0, 7, 5), (4, 3, 50257, 700, 300, 0.75, 0, 0),
          (8, 2, 131072, 2000, 1024, 0.75, 8, 0), (1, 600, 300, 3, 1, 0.1, 0, 0), (2, 3, 40000, 0, 0, 0.9, 0, 2), (1, 4, 3000, 50, 0, None, 0, 0)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("W,T,V,L,K,masked,pad,offset", SHAPES)
def test_adjust(mr, W, T, V, L, K, masked, pad, offset, dtype, in_place):
    _check(mr, _scores(T, V, dtype, 1), dtype, W, _lists(T, V, L, K, masked, 2), pad, offset, in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("W,T,V,L,K,masked,pad,offset", SHAPES)
def test_gradient(mr, W, T, V, L, K, masked, pad, offset, dtype, in_place):
    _check_grad(mr, _scores(T, V, dtype, 1), dtype, W, _lists(T, V, L, K, masked, 2), pad, offset, in_place)


@pytest.mark.parametrize("which", ["repetition", "frequency", "presence"])
def test_one_penalty_at_a_time(mr, which):
    a = _lists(5, 777, 60, 0, None, 4)
    a = {k: v for k, v in a.items() if k in ("history", which)}
    _check(mr, _scores(5, 777, "bf16", 3), "bf16", 2, a)
    _check_grad(mr, _scores(5, 777, "bf16", 3), "bf16", 2, a)
    a["n_prompt"] = a["history"].new_tensor([0, 60, 30, 70, -1])
    _check(mr, _scores(5, 777, "fp32", 3), "fp32", 2, a)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("in_place", [False, True])
def test_odd_values(mr, dtype, in_place):
    """Infinities, NaN and the type's lowest value, masked and not, listed and not."""
    import torch
    T, V = 4, 600
    x = _scores(T, V, dtype, 5)
    low = torch.finfo(_dt(dtype)).min
    for i, v in enumerate([INF, -INF, float("nan"), low, -low, -0.0, 1e-40]):
        x[:, 10 * i:10 * i + 5] = v
    a = _lists(T, V, 200, 50, 0.5, 6)
    a["mask"][0] = 0                # a row that allows nothing
    a["mask"][1] = -1               # all
    a["bias"][:, 3] = -INF          # a banned token
    a["bias_ids"][:, 3] = 300
    _check(mr, x, dtype, 1, a, in_place=in_place)
    _check_grad(mr, x, dtype, 3, a, in_place=in_place)


def test_masked_places_are_not_looked_at(mr):
    import torch
    T, V = 3, 4096
    x = torch.full((T, V), float("nan"))
    x[:, ::64] = 1.0
    mask = torch.zeros(T, V // 32, dtype=torch.int32)
    mask[:, ::2] = 1
    for dtype in ("fp32", "bf16"):
        _check(mr, x.to(_dt(dtype)), dtype, 2, {"mask": mask})


def test_long_counts(mr):
    """One token all along the history: counts that 16 bits could not hold."""
    import torch
    T, V, L = 2, 500, 100000
    h = torch.full((T, L), 123)
    h[1, ::2] = 7
    a = {"history": h, "frequency": torch.tensor([1e-3, 2e-3]), "presence": torch.tensor([0.5, -0.25])}
    _check(mr, _scores(T, V, "fp32", 1), "fp32", 1, a)


@pytest.mark.parametrize("L,K", [(8447, 1), (8448, 0), (7500, 948), (8448, 1), (20000, 0), (9000, 1024)])
def test_long_histories(mr, L, K):
    """Both sides of the longest list of which a wide window may name every entry, each entry another token."""
    import torch
    T, V = 2, 70001
    g = torch.Generator().manual_seed(L)
    a = _lists(T, V, L, K, 0.3, 11)
    a["history"] = torch.stack([torch.randperm(V, generator=g)[:L] for _ in range(T)])
    a["n_history"], a["n_prompt"] = torch.tensor([L, L]), torch.tensor([L // 3, 0])
    # a window whose every column is named
    a["history"][1] = (torch.arange(L) + 8192) % V
    _check(mr, _scores(T, V, "bf16", 1), "bf16", 2, a)
    _check(mr, _scores(T, V, "fp32", 1), "fp32", 1, a, in_place=True)
    _check_grad(mr, _scores(T, V, "bf16", 1), "bf16", 1, a)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_sides_on_other_boundaries(mr, dtype):
    """Rows of the output elsewhere past a 16-byte boundary than the scores'."""
    import torch
    T, V = 3, 9001
    x = _scores(T, V, dtype, 1)
    a = _lists(T, V, 300, 9, 0.4, 12)
    logits, out = Shards(2, x, 3, 1), Shards(2, torch.zeros_like(x), 0, 2)
    same = Shards(2, torch.zeros_like(x), 3, 1)
    mr.mr_adjust_logits(logits.views, out.views, **_cuda(a))
    mr.mr_adjust_logits(logits.views, same.views, **_cuda(a))
    torch.cuda.synchronize()
    assert torch.equal(out.host(), same.host())
    out.fenced()


def test_calls_side_by_side(mr):
    """Two streams at once, other rows and lists on each."""
    import torch
    calls = []
    for k in range(2):
        x = _scores(40, 30011, "bf16", k).cuda()
        a = _cuda(_lists(40, 30011, 500 + 100 * k, 8, 0.2, k))
        want, out = torch.empty_like(x), torch.empty_like(x)
        mr.mr_adjust_logits([x], [want], **a)
        calls.append((x, a, want, out, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for x, a, _, out, stream in calls:
            mr.mr_adjust_logits([x], [out], stream=stream, **a)
    torch.cuda.synchronize()
    for _, _, want, out, _ in calls:
        assert torch.equal(out, want)


def test_column_slices_of_one_buffer(mr):
    import torch
    T, V, W = 4, 1003, 3
    x = _scores(T, V, "bf16", 8)
    a = _lists(T, V, 90, 11, 0.4, 9)
    cuts = [r * V // W for r in range(W + 1)]
    flat, out = x.cuda(), torch.empty(T, V + 5, dtype=torch.bfloat16, device="cuda")
    mr.mr_adjust_logits([flat[:, lo:hi] for lo, hi in zip(cuts, cuts[1:])], [out[:, lo:hi] for lo, hi in zip(cuts, cuts[1:])], **_cuda(a))
    whole = torch.empty(T, V, dtype=torch.bfloat16, device="cuda")
    mr.mr_adjust_logits([flat], [whole], **_cuda(a))
    assert torch.equal(out[:, :V], whole)


def test_some_ranks_beside_one_another(mr):
    """Ranks 0 and 1 of a buffer, 2 and 3 of buffers of their own, 4 behind 5's place, one rank without a column before them."""
    import torch
    T, V, W = 3, 5, 6           # cuts 0 0 1 2 3 4 5
    for V in (5, 6007):
        x = _scores(T, V, "fp32", 8).cuda()
        a = _lists(T, V, 60, 5, 0.4, 9)
        cuts = [r * V // W for r in range(W + 1)]
        one, two = torch.zeros(T, V + 9, device="cuda"), torch.zeros(T, V + 9, device="cuda")
        xs, outs = [], []
        for r in range(W):
            lo, hi = cuts[r], cuts[r + 1]
            if r in (2, 3):
                src, dst = torch.empty(T, hi - lo, device="cuda"), torch.empty(T, hi - lo, device="cuda")
            elif r == 4:
                src, dst = one[:, lo:hi], torch.empty(T, hi - lo, device="cuda")
            else:
                src, dst = one[:, lo:hi], two[:, lo:hi]
            src.copy_(x[:, lo:hi])
            xs.append(src)
            outs.append(dst)
        whole = torch.empty_like(x)
        mr.mr_adjust_logits(xs, outs, **_cuda(a))
        mr.mr_adjust_logits([x], [whole], **_cuda(a))
        assert torch.equal(torch.cat(outs, 1), whole)
        back = {k: v for k, v in _cuda(a).items() if not k.startswith("bias")}
        g = _scores(T, V, "fp32", 3).cuda()
        mr.mr_adjust_logits_grad(xs, [g[:, lo:hi] for lo, hi in zip(cuts, cuts[1:])], outs, **back)
        mr.mr_adjust_logits_grad([x], [g], [whole], **back)
        assert torch.equal(torch.cat(outs, 1), whole)


def test_gradient_against_differences(mr):
    """Central differences of the adjusted scores themselves; no score lies so near 0 that a step crosses it."""
    import torch
    T, V, step = 3, 40, 2.0 ** -6
    x = _scores(T, V, "fp32", 3)
    x = torch.where(x.abs() < 0.1, torch.full_like(x, 0.5), x)
    a = _cuda(_lists(T, V, 30, 6, 0.3, 4))
    g = torch.randn(T, V, generator=torch.Generator().manual_seed(1))
    grad = torch.empty(T, V, device="cuda")
    mr.mr_adjust_logits_grad([x.cuda()], [g.cuda()], [grad], **{k: v for k, v in a.items() if not k.startswith("bias")})
    up, down = torch.empty(T, V, device="cuda"), torch.empty(T, V, device="cuda")
    mr.mr_adjust_logits([(x + step).cuda()], [up], **a)
    mr.mr_adjust_logits([(x - step).cuda()], [down], **a)
    d = (up.double() - down.double()).cpu() / (2 * step)       # a column's score depends on that column alone
    d = torch.where(torch.isfinite(up.cpu()), d, torch.zeros_like(d))
    # either side: x +- step, and each of four steps, rounded, of values below 64
    assert float((grad.double().cpu() - d * g.double()).abs().max()) < 2 * 5 * 64 * 2.0 ** -24 / (2 * step) * 4


def test_far_rows(mr):
    """Rows more than 2^32 elements from the first."""
    import torch
    V, ld = 70, 1 << 30
    buf = torch.zeros(4 * ld + V, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (5, V), (ld, 1))
    x.fill_(2.0)
    a = {"history": torch.full((5, 1), 69), "repetition": torch.full((5,), 4.0), "mask": torch.full((5, 3), -2, dtype=torch.int32)}
    mr.mr_adjust_logits([x], [x], **_cuda(a))
    assert bool((x[:, 69] == 0.5).all()) and bool((x[:, 0] == -INF).all()) and bool((x[:, 64] == -INF).all())
    assert bool((x[:, 65:69] == 2.0).all()) and bool((buf[V:ld] == 0).all())


def test_streams_and_graphs(mr):
    import torch
    T, V, W = 6, 5003, 2
    x = _scores(T, V, "bf16", 3).cuda()
    a = _cuda(_lists(T, V, 100, 9, 0.5, 4))
    cut = V // W
    split = lambda t: [t[:, :cut], t[:, cut:]]  # noqa: E731
    want, out = torch.empty_like(x), torch.empty_like(x)
    mr.mr_adjust_logits(split(x), split(want), **a)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    mr.mr_adjust_logits(split(x), split(out), stream=side, **a)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mr.mr_adjust_logits(split(x), split(out), **a)
        mr.mr_adjust_logits_grad(split(x), split(out), split(out), **{k: v for k, v in a.items() if not k.startswith("bias")})
    for seed in (7, 8):
        b = _cuda(_lists(T, V, 100, 9, 0.5, seed))
        for k, v in a.items():
            v.copy_(b[k])
        graph.replay()
        mr.mr_adjust_logits(split(x), split(want), **a)
        mr.mr_adjust_logits_grad(split(x), split(want), split(want), **{k: v for k, v in a.items() if not k.startswith("bias")})
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_no_rows(mr):
    import torch
    x = torch.empty(0, 10, device="cuda")
    mr.mr_adjust_logits([x], [x])
    mr.mr_adjust_logits_grad([x], [x], [x])
    y = torch.randn(3, 10, device="cuda")
    z = torch.empty_like(y)
    mr.mr_adjust_logits([y], [z])       # nothing to adjust: a copy
    assert torch.equal(y, z)
    mr.mr_adjust_logits([y], [z], history=torch.empty(3, 0, dtype=torch.int64, device="cuda"), repetition=torch.ones(3, device="cuda"))
    assert torch.equal(y, z)
