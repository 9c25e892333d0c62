"""The embedding lookup and its gradient against their definitions, at the
sizes, layouts and ids where they can go wrong.

The lookup is one fp32 product rounded once: it has the bits of the same two
steps by torch.  The gradient's bounds are derived in step_ref.embedding_grad;
the rounding to its type adds half a step."""
import numpy as np
import pytest

import step_ref as ref

pytestmark = pytest.mark.gpu


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


class Block:
    """[rows, n] inside a fenced allocation: `pad` elements between rows, `offset` before the first."""

    FENCE = 64

    def __init__(self, rows, n, dtype, pad=0, offset=0, fill=None):
        import torch
        self.raw = torch.full((rows * (n + pad) + offset + 2 * self.FENCE,), 77.0, dtype=_dt(dtype), device="cuda")
        self.view = torch.as_strided(self.raw, (rows, n), (n + pad, 1), self.FENCE + offset)
        if fill is not None:
            self.view.copy_(fill)

    def fenced(self):
        keep = self.raw.clone()
        keep.as_strided(self.view.shape, self.view.stride(), self.view.storage_offset()).fill_(77.0)
        assert bool((keep == 77.0).all()), "written outside the rows"


def _cuts(V, W):
    return [r * V // W for r in range(W + 1)]


def _table(W, V, H, dtype, pad, offset, fill=None):
    cuts = _cuts(V, W)
    return [Block(hi - lo, H, dtype, pad, offset, None if fill is None else fill[lo:hi]) for lo, hi in zip(cuts, cuts[1:])]


def _random(shape, dtype, seed):
    import torch
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(_dt(dtype))


def _ids(T, V, seed, kind="mixed"):
    import torch
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        return torch.full((T,), V - 1)
    if kind == "two":
        return torch.where(torch.rand(T, generator=g) < 0.9, 0, V - 1)
    if kind == "none":
        return torch.full((T,), -1)
    ids = torch.randint(0, V, (T,), generator=g)
    often = torch.rand(T, generator=g)
    ids[often < 0.3] = 0
    ids[(often > 0.3) & (often < 0.4)] = V // 2
    if kind == "mixed" and T > 3:
        ids[torch.randint(0, T, (T // 8 + 1,), generator=g)] = -100
        ids[1], ids[2] = V, -2 ** 63
    return ids


# (W, T, V, H, pad, offset): one of each, fewer rows than ranks, odd row lengths, rows off
# every boundary, both sides of a vector, of a warp's part and of a slab
SHAPES = [(1, 1, 1, 1, 0, 0), (2, 5, 1, 8, 0, 0), (64, 40, 63, 16, 0, 0), (8, 33, 5, 7, 3, 1), (1, 7, 100, 255, 0, 0), (3, 64, 50, 256, 0, 0),
          (1, 65, 1000, 257, 0, 3), (4, 200, 301, 512, 8, 0), (1, 31, 4000, 1001, 0, 0), (2, 300, 77, 1024, 8, 8), (1, 9, 33, 1032, 0, 0),
          (5, 1000, 10007, 64, 1, 0), (1, 3, 12, 8200, 0, 0), (1, 2049, 700, 24, 0, 0)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("W,T,V,H,pad,offset", SHAPES)
def test_lookup(mr, W, T, V, H, pad, offset, dtype):
    import torch
    table = _random((V, H), dtype, 1)
    ids = _ids(T, V, 2)
    for scale in (1.0, -0.3):
        shards, out = _table(W, V, H, dtype, pad, offset, table), Block(T, H, dtype, pad, offset)
        mr.mr_embedding([s.view for s in shards], ids.cuda(), out.view, scale=scale)
        torch.cuda.synchronize()
        there = (ids >= 0) & (ids < V)
        want = (table[ids.clamp(0, V - 1)].float() * scale).to(_dt(dtype))
        want[~there] = torch.where(ids[~there] < 0, 0.0, float("nan"))[:, None].to(_dt(dtype))
        assert torch.equal(out.view.cpu().nan_to_num(99.0), want.nan_to_num(99.0))
        out.fenced()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_lookup_at_every_place(mr, dtype):
    """Rows of the table and of the output at every place past a 16-byte boundary, rows of one vector to a few."""
    import torch
    lanes = 8 if dtype == "bf16" else 4
    for H in list(range(1, 5 * lanes)) + [511, 1030]:
        table = _random((9, H), dtype, H)
        ids = torch.tensor([3, 0, 8, -1, 5, 9, 7])
        want = (table[ids.clamp(0, 8)].float() * 1.5).to(_dt(dtype))
        want[3], want[5] = 0.0, float("nan")
        for a in range(lanes):
            shard, out = Block(9, H, dtype, 1, a, table), Block(7, H, dtype, 2, (3 * a + H) % lanes)
            mr.mr_embedding([shard.view], ids.cuda(), out.view, scale=1.5)
            assert torch.equal(out.view.cpu().nan_to_num(99.0), want.nan_to_num(99.0)), (H, a)
            out.fenced()


def test_lookup_keeps_infinities(mr):
    import torch
    for dtype in ("fp32", "bf16"):
        table = _random((4, 16), dtype, 1)
        table[0, 3], table[1, 2], table[2, 1], table[3, 0] = float("inf"), float("-inf"), float("nan"), 3e38
        out = torch.empty(4, 16, dtype=_dt(dtype), device="cuda")
        mr.mr_embedding([table.cuda()], torch.arange(4, device="cuda"), out, scale=2.0)
        want = (table.float() * 2.0).to(_dt(dtype))
        assert torch.equal(out.cpu().nan_to_num(99.0, 1e38, -1e38), want.nan_to_num(99.0, 1e38, -1e38))


def _check_grad(mr, W, T, V, H, pad, offset, dtype, table, accumulate, kind="mixed", scale=1.5, seed=3):
    import torch
    g = _random((T, H), dtype, seed)
    ids = _ids(T, V, seed + 1, kind)
    old = _random((V, H), table, seed + 2)
    # rows of g_out that no token reads hold NaN
    dead = (ids < 0) | (ids >= V)
    g_in = g.clone()
    g_in[dead] = float("nan")
    x, shards = Block(T, H, dtype, pad, offset, g_in), _table(W, V, H, table, pad, offset, old if accumulate else torch.full((V, H), 7.0))
    mr.mr_embedding_grad(x.view, ids.cuda(), [s.view for s in shards], scale=scale, accumulate=accumulate)
    torch.cuda.synchronize()
    got = torch.cat([s.view.cpu() for s in shards])
    want, bound, untouched = ref.embedding_grad(g.double().numpy(), ids.numpy(), V, scale, old.double().numpy() if accumulate else None)
    ref.close(got.double().numpy(), want, bound + np.where(untouched[:, None], 0.0, ref.rounded(want, table)), "gradient")
    if accumulate:
        assert torch.equal(got[torch.from_numpy(untouched)], old[torch.from_numpy(untouched)])
    for s in shards:
        s.fenced()
    return got


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype,table", [("fp32", "fp32"), ("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("W,T,V,H,pad,offset", SHAPES)
def test_gradient(mr, W, T, V, H, pad, offset, dtype, table, accumulate):
    _check_grad(mr, W, T, V, H, pad, offset, dtype, table, accumulate)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("kind", ["one", "two", "none", "plain"])
@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 64, 65, 97, 1000, 1023, 1024, 1025, 4096, 5000])
def test_gradient_of_crowded_tokens(mr, T, kind, accumulate):
    _check_grad(mr, 2, T, 129, 40, 0, 0, "bf16", "fp32", accumulate, kind)


@pytest.mark.parametrize("T", [9000, 20011, 70001])
@pytest.mark.parametrize("kind", ["one", "two", "mixed"])
def test_gradient_of_many_tokens(mr, T, kind):
    _check_grad(mr, 3, T, 40009, 17, 0, 0, "bf16", "fp32", False, kind)
    _check_grad(mr, 1, T, 1 << 17, 16, 0, 0, "bf16", "bf16", True, kind)


@pytest.mark.parametrize("T", [131072, 131073, 262144])
def test_gradient_of_the_most_tokens(mr, T):
    """Sums of whole numbers, exact in fp32."""
    import torch
    V, H = 50021, 8
    ids = _ids(T, V, 5).cuda()
    g = torch.randint(-8, 9, (T, H), generator=torch.Generator().manual_seed(1)).float().cuda()
    grad = torch.empty(V, H, device="cuda")
    mr.mr_embedding_grad(g, ids, [grad])
    on = (ids >= 0) & (ids < V)
    want = torch.zeros(V, H, dtype=torch.float64, device="cuda").index_add_(0, ids[on], g[on].double())
    assert torch.equal(grad.double(), want)


def test_gradient_of_more_rows_than_a_call_takes(mr):
    import torch
    T = 262145
    with pytest.raises(mr.MRError, match="UNSUPPORTED"):
        mr.mr_embedding_grad(torch.zeros(T, 1, device="cuda"), torch.zeros(T, dtype=torch.int64, device="cuda"), [torch.zeros(1, 1, device="cuda")])


@pytest.mark.parametrize("V", [1, 2, 3, 31, 32, 1023, 1024, (1 << 20) - 1, 1 << 20, (1 << 20) + 1])
def test_gradient_of_vocabularies_at_the_sort_digits(mr, V):
    import torch
    T, H = 3000, 4
    ids = _ids(T, V, V).cuda()
    ids[5] = V - 1
    g = torch.randint(-8, 9, (T, H), generator=torch.Generator().manual_seed(1)).float().cuda()
    grad = torch.empty(V, H, device="cuda")
    mr.mr_embedding_grad(g, ids, [grad])
    on = (ids >= 0) & (ids < V)
    want = torch.zeros(V, H, dtype=torch.float64, device="cuda").index_add_(0, ids[on], g[on].double())
    assert torch.equal(grad.double(), want)


def test_gradients_side_by_side(mr):
    """Two streams at once, a workspace each."""
    import torch
    calls = []
    for k in range(2):
        T, V, H = 3000 + 1000 * k, 7001, 264
        g, ids = _random((T, H), "bf16", k).cuda(), _ids(T, V, k).cuda()
        want, grad = torch.empty(V, H, device="cuda"), torch.empty(V, H, device="cuda")
        mr.mr_embedding_grad(g, ids, [want])
        work = torch.empty(mr.mr_embedding_grad_workspace_bytes(T, V, H), dtype=torch.uint8, device="cuda")
        calls.append((g, ids, want, grad, work, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for g, ids, _, grad, work, stream in calls:
            mr.mr_embedding_grad(g, ids, [grad], workspace=work, stream=stream)
    torch.cuda.synchronize()
    for _, _, want, grad, _, _ in calls:
        assert torch.equal(grad, want)


def test_gradient_without_tokens(mr):
    import torch
    grad = torch.ones(10, 8, device="cuda")
    ids, g = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, 8, device="cuda")
    mr.mr_embedding_grad(g, ids, [grad], accumulate=True)
    assert bool((grad == 1).all())
    mr.mr_embedding_grad(g, ids, [grad])
    assert bool((grad == 0).all())
    mr.mr_embedding([grad], ids, torch.empty(0, 8, device="cuda"))


def test_gradient_against_differences(mr):
    """The gradient of a weighted sum of the looked-up rows, by central differences of the lookup itself."""
    import torch
    V, H, T, scale = 7, 5, 12, 0.5
    table = _random((V, H), "fp32", 1).cuda()
    ids = torch.tensor([0, 1, 1, 6, -1, 3, 0, 0, 5, 6, 6, 1], device="cuda")
    w = _random((T, H), "fp32", 2).cuda()
    grad = torch.empty(V, H, device="cuda")
    mr.mr_embedding_grad(w, ids, [grad], scale=scale)
    out = torch.empty(T, H, device="cuda")

    def value(t):
        mr.mr_embedding([t], ids, out, scale=scale)
        return float((out.double() * w.double()).sum())

    step = 0.25         # the sum is linear in the table: no step is too wide
    for v in range(V):
        for c in range(H):
            up, down = table.clone(), table.clone()
            up[v, c] += step
            down[v, c] -= step
            d = (value(up) - value(down)) / (2 * step)
            # both values: rounded table entries and products, U each of |scale x w|
            assert abs(d - float(grad[v, c])) < 12 * 4 * 2.0 ** -24 * 16 / step


def test_gradient_is_the_same_on_every_run(mr):
    import torch
    T, V, H = 30000, 5000, 72
    g, ids = _random((T, H), "bf16", 1).cuda(), _ids(T, V, 2).cuda()
    first = None
    for _ in range(5):
        grad = torch.empty(V, H, device="cuda")
        mr.mr_embedding_grad(g, ids, [grad])
        first = grad if first is None else first
        assert torch.equal(first, grad)


def test_row_slices_of_one_buffer(mr):
    import torch
    V, H, W, T = 1001, 64, 4, 500
    cuts = _cuts(V, W)
    table = _random((V, H + 16), "bf16", 1).cuda()
    shards = [table[lo:hi, 8:8 + H] for lo, hi in zip(cuts, cuts[1:])]
    ids = _ids(T, V, 2, "plain").cuda()
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    mr.mr_embedding(shards, ids, out)
    assert torch.equal(out, table[ids][:, 8:8 + H])


def test_far_rows(mr):
    """Offsets past 2^32 bytes and elements: of the table, of the rows, and of a stride."""
    import torch
    V, H = 5, 1 << 30
    table = torch.zeros(V, H, dtype=torch.bfloat16, device="cuda")
    table[4, -8:] = 3.0
    out = torch.full((2, H), 9.0, dtype=torch.bfloat16, device="cuda")
    mr.mr_embedding([table], torch.tensor([0, 4], device="cuda"), out, scale=2.0)
    assert float(out[0, -1]) == 0.0 and float(out[1, -1]) == 6.0 and float(out[1, -9]) == 0.0
    mr.mr_embedding_grad(out, torch.tensor([4, 4], device="cuda"), [table], accumulate=True)
    assert float(table[4, -1]) == 9.0 and float(table[4, 0]) == 0.0 and float(table[3, -1]) == 0.0
    del table, out
    wide = torch.zeros(5, 1 << 30, dtype=torch.bfloat16, device="cuda")[:, :24]
    wide[4] = 1.5
    out = torch.empty(1, 24, dtype=torch.bfloat16, device="cuda")
    mr.mr_embedding([wide], torch.tensor([4], device="cuda"), out)
    assert bool((out == 1.5).all())


def test_streams_and_graphs(mr):
    import torch
    T, V, H = 300, 2000, 96
    table, g = _random((V, H), "bf16", 1).cuda(), _random((T, H), "bf16", 2).cuda()
    ids = _ids(T, V, 3).cuda()
    out, want = torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    grad, want_grad = torch.empty(V, H, device="cuda"), torch.empty(V, H, device="cuda")
    mr.mr_embedding([table], ids, want)
    mr.mr_embedding_grad(g, ids, [want_grad])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        out.zero_()
        grad.fill_(5.0)
        torch.cuda.synchronize()
        mr.mr_embedding([table], ids, out, stream=stream)
        mr.mr_embedding_grad(g, ids, [grad], stream=stream)
        side.synchronize()
        assert torch.equal(out.nan_to_num(9.0), want.nan_to_num(9.0)) and torch.equal(grad, want_grad)
    # captured, with the ids changed between replays
    work = torch.empty(max(16, mr.mr_embedding_grad_workspace_bytes(T, V, H)), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mr.mr_embedding([table], ids, out)
        mr.mr_embedding_grad(g, ids, [grad], workspace=work)
    for seed in (5, 6):
        ids.copy_(_ids(T, V, seed))
        work.fill_(255)
        graph.replay()
        mr.mr_embedding([table], ids, want)
        mr.mr_embedding_grad(g, ids, [want_grad])
        torch.cuda.synchronize()
        assert torch.equal(out.nan_to_num(9.0), want.nan_to_num(9.0)) and torch.equal(grad, want_grad)
