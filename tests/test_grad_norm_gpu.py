"""The gradient norm and the clipping against their definitions.

Bounds, from the arithmetic (U = 2^-24): a product is off by U, a thread's sum
of up to 64 terms of one sign by 64 U, the sums of those are kept in pairs of
floats and joined in 64 bits.  A norm has half of that, and its rounding: 34 U.
A clipped value has the norm's 34 U in its factor, that factor's rounding and its
own, and half a step of its type."""
import numpy as np
import pytest

import step_ref as ref

pytestmark = pytest.mark.gpu
U = ref.U
NORM = 34 * U
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


def _tensors(sizes, dtypes, seed=0, scale=1.0, offset=0):
    """Tensors inside one fenced buffer a type, `offset` elements off the 256-byte boundaries."""
    import torch
    g = torch.Generator().manual_seed(seed)
    out = []
    for n, d in zip(sizes, dtypes):
        raw = torch.full((n + 160,), 77.0, dtype=_dt(d), device="cuda")
        v = raw[64 + offset:64 + offset + n]
        v.copy_((torch.randn(n, generator=g) * scale).to(_dt(d)))
        out.append((raw, v))
    return out


def _fenced(pairs):
    for raw, v in pairs:
        keep = raw.clone()
        keep[v.storage_offset():v.storage_offset() + v.numel()] = 77.0
        assert bool((keep == 77.0).all()), "written outside the tensor"


def _host(ts):
    return [t.double().cpu().numpy() for t in ts]


def _check(mr, ts, dtypes, max_norm, out_offset=0, in_place=False):
    import torch
    host = _host(ts)
    want = ref.norm(host)
    norm = torch.full((1,), 77.0, device="cuda")
    mr.mr_grad_norm(ts, norm)
    with np.errstate(over="ignore"):
        rounded = np.float64(np.float32(want))
    ref.close([float(norm)], [rounded], NORM * (want if np.isfinite(want) else 0) + 2.0 ** -149, "norm")
    first = float(norm)
    pairs = [(None, t) for t in ts] if in_place else _tensors([t.numel() for t in ts], dtypes, 9, offset=out_offset)
    outs = [v for _, v in pairs]
    norm.fill_(77.0)
    mr.mr_clip_grad_norm(ts, outs, max_norm, norm=norm)
    torch.cuda.synchronize()
    assert np.float32(first).tobytes() == np.float32(float(norm)).tobytes() or first != first
    with np.errstate(all="ignore"):
        coef = 1.0 if want <= max_norm else max_norm / want
    near = abs(want - max_norm) <= NORM * want if np.isfinite(want) else False
    for d, h, o in zip(dtypes, host, outs):
        with np.errstate(all="ignore"):
            w = h * coef
        off = np.where(np.isfinite(w), np.abs(w), 0.0) * (0 if coef == 1.0 and not near else NORM + 3 * U) * 1.01
        ref.close(o.double().cpu().numpy(), w, off + (0 if coef == 1.0 and not near else ref.rounded(w, d)), "clipped")
    if not in_place:
        _fenced(pairs)
        for h, t in zip(host, ts):
            assert np.array_equal(t.double().cpu().numpy(), h, equal_nan=True)


SIZES = [[1], [3, 0, 5], [4095], [4096], [4097], [8191, 8192, 8193], [1, 2, 3, 4, 5, 6, 7, 8, 9], [100000, 1, 33, 70000], [2000003], [300] * 40]


@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("types", ["fp32", "bf16", "mixed"])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: str(sum(s)))
def test_norm_and_clip(mr, sizes, types, offset):
    dtypes = [types if types != "mixed" else ("fp32", "bf16")[i % 2] for i in range(len(sizes))]
    ts = [v for _, v in _tensors(sizes, dtypes, 1, offset=offset)]
    for max_norm in (0.25, 1e9, 0.0, INF):
        _check(mr, ts, dtypes, max_norm, out_offset=offset)
    _check(mr, ts, dtypes, 0.5, out_offset=2)       # out off the gradient's boundary
    _check(mr, ts, dtypes, 0.5, in_place=True)


@pytest.mark.parametrize("count", [511, 512, 513, 1500])
def test_long_lists(mr, count):
    import torch
    flat = torch.randn(count * 40, generator=torch.Generator().manual_seed(1)).cuda()
    ts = [flat[40 * i:40 * i + 37 - i % 3] for i in range(count)]
    _check(mr, ts, ["fp32"] * count, 2.0)
    _check(mr, ts, ["fp32"] * count, 2.0, in_place=True)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-20, 2.0 ** -30, 1e-10, 1e10, 2.0 ** 61, 1e25, 1e36])
def test_range(mr, dtype, scale):
    """Squares far outside fp32's range, in one tile and in many."""
    for n in (5, 3001, 300000):
        ts = [v for _, v in _tensors([n], [dtype], 2, scale)]
        _check(mr, ts, [dtype], scale)


def test_values_of_every_size_together(mr):
    import torch
    g = torch.Generator().manual_seed(3)
    for top in (-30, 0, 30, 100):
        x = torch.randn(50000, generator=g) * 2.0 ** (top - 120 * torch.rand(50000, generator=g))
        _check(mr, [x.cuda()], ["fp32"], 2.0 ** (top - 3))


def test_norm_beyond_fp32(mr):
    """The norm reads +inf, and what is clipped comes from the norm itself."""
    import torch
    x = torch.full((1 << 20,), 3e38, device="cuda")
    norm, out = torch.empty(1, device="cuda"), torch.empty_like(x)
    mr.mr_clip_grad_norm([x], [out], 1024.0, norm=norm)
    assert float(norm) == INF
    assert abs(float(out[7]) - 1.0) < 1e-6 and bool((out == out[0]).all())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_nothing_and_no_numbers(mr, dtype):
    import torch
    norm = torch.full((1,), 7.0, device="cuda")
    mr.mr_grad_norm([], norm)
    assert float(norm) == 0.0
    mr.mr_clip_grad_norm([], [], 1.0, norm=norm.fill_(7.0))
    assert float(norm) == 0.0
    mr.mr_clip_grad_norm([], [], 1.0)
    _check(mr, [torch.zeros(5000, dtype=_dt(dtype), device="cuda"), torch.empty(0, dtype=_dt(dtype), device="cuda")], [dtype] * 2, 0.0)
    for bad in (float("nan"), INF, -INF):
        for at in (0, 4999, 20000):
            x = torch.randn(20001, generator=torch.Generator().manual_seed(1)).to(_dt(dtype)).cuda()
            x[at] = bad
            _check(mr, [x], [dtype], 1.0)
    x = torch.tensor([INF, float("nan"), 1.0], dtype=_dt(dtype), device="cuda")
    _check(mr, [x], [dtype], 1.0)


def test_a_tensor_listed_twice(mr):
    import torch
    x = torch.randn(1000, device="cuda")
    norm = torch.empty(1, device="cuda")
    mr.mr_grad_norm([x, x], norm)
    want = float((2 * x.double().square().sum()).sqrt())
    assert abs(float(norm) - want) <= NORM * want
    with pytest.raises(mr.MRError, match="ALIAS"):
        mr.mr_clip_grad_norm([x, x], [x, x], 1.0)


def test_many_elements(mr):
    """More than 2^32 elements in one tensor, the last of them the only large one."""
    import torch
    x = torch.zeros((1 << 32) + 4099, dtype=torch.bfloat16, device="cuda")
    x[-1] = 3.0
    x[5] = 4.0
    norm = torch.empty(1, device="cuda")
    mr.mr_clip_grad_norm([x], [x], 1.0, norm=norm)
    assert float(norm) == 5.0
    assert float(x[-1]) == float(torch.tensor(0.6).bfloat16()) and float(x[5]) == float(torch.tensor(0.8).bfloat16()) and float(x[-2]) == 0.0


def test_the_same_on_every_run(mr):
    import torch
    x = [torch.randn(n, generator=torch.Generator().manual_seed(n)).cuda() for n in (1000003, 77, 500000)]
    norm = torch.empty(1, device="cuda")
    seen = set()
    for _ in range(5):
        mr.mr_grad_norm(x, norm)
        seen.add(float(norm))
    assert len(seen) == 1


def test_host_threads(mr):
    """Threads at once on one stream and on streams of their own, without workspaces of the caller's."""
    import threading

    import torch
    lists = [[torch.randn(n, generator=torch.Generator().manual_seed(n)).cuda() * (k + 1) for n in (70001, 300, 5000)] for k in range(4)]
    wants = [ref.norm(_host(x)) for x in lists]
    streams = [torch.cuda.current_stream()] * 2 + [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    bad = []

    def work(k):
        with torch.cuda.stream(streams[k]):
            norms = [torch.empty(1, device="cuda") for _ in range(200)]
            for n in norms:
                mr.mr_grad_norm(lists[k], n)
            streams[k].synchronize()
            bad.extend(float(n) for n in norms if not abs(float(n) - wants[k]) <= NORM * wants[k])

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_two_graphs_and_calls_between(mr):
    """Graphs captured without the caller's workspace, replayed on two streams beside calls on a third."""
    import torch
    lists = [[torch.randn(n, generator=torch.Generator().manual_seed(n + k)).cuda() for n in (200000, 77, 3000)] for k in range(3)]
    wants = [ref.norm(_host(x)) for x in lists]
    norms = [torch.zeros(1, device="cuda") for _ in range(3)]
    graphs = []
    for k in range(2):
        mr.mr_grad_norm(lists[k], norms[k])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mr.mr_grad_norm(lists[k], norms[k])
        graphs.append((g, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(30):
        for g, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
        mr.mr_grad_norm(lists[2], norms[2])
    torch.cuda.synchronize()
    for n, w in zip(norms, wants):
        assert abs(float(n) - w) <= NORM * w


def test_streams_and_graphs(mr):
    import torch
    x = [torch.randn(n, device="cuda") for n in (5000, 12, 70000)]
    out = [torch.empty_like(t) for t in x]
    norm = torch.zeros(1, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        norm.zero_()
        torch.cuda.synchronize()
        mr.mr_clip_grad_norm(x, out, 1.0, norm=norm, stream=stream)
        side.synchronize()
        want = ref.norm(_host(x))
        assert abs(float(norm) - want) <= NORM * want
    work = torch.empty(mr.mr_grad_norm_workspace_bytes(3), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mr.mr_clip_grad_norm(x, x, 1.0, norm=norm, workspace=work)
    for t in x:
        t.normal_()
    before = ref.norm(_host(x))
    work.fill_(255)
    graph.replay()
    torch.cuda.synchronize()
    assert abs(float(norm) - before) <= NORM * before
    graph.replay()      # clipped in place: the second replay finds a norm of 1
    torch.cuda.synchronize()
    assert abs(float(norm) - 1.0) <= 1e-5
