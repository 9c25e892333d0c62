"""The gradient norm and the clipping where their sums could lose something:
many elements, and more than 2^32 of the largest.

Bounds, from the arithmetic (U = 2^-24, half an fp32 step of 1).  Elements come
in pairs a, b: the square of a is rounded (exact for bf16, whose squares have 16
bits), a fused multiply-add with b rounds once more.  Pairs are added without
loss to two floats, whose second loses less than 2^-38 of the sum.  So a sum of
terms of one sign is off by 2 U for fp32 and U for bf16, its root by half of
that, and the root's rounding is half a step of the norm.  Where all pairs are
exact, that half step is all."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


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


def test_most_of_the_largest(mr):
    """2^33 elements of bf16's largest value: the norm, 2^16.5 times that, reads
    +inf, and the factor still comes from the norm itself."""
    import torch
    n, x, most = 1 << 33, 255 * 2.0 ** 120, 2.0 ** 60
    t = torch.full((n,), x, dtype=torch.bfloat16, device="cuda")
    norm = torch.zeros(1, device="cuda")
    mr.mr_clip_grad_norm([t], [t], most, norm=norm)
    assert float(norm) == float("inf")
    # most / 2^16.5, rounded to bf16: 1.41421 * 2^43 lies 0.0038 of itself from the nearest
    # point between two bf16 values, which the factor's few U do not reach
    want = torch.tensor(most / 2 ** 16.5, dtype=torch.float64).bfloat16()
    wrong = sum(int((part != want.cuda()).sum()) for part in t.split(1 << 30))
    assert wrong == 0


def _half_step(v):
    return float(np.spacing(np.float32(v))) / 2


def _norm64(ts):
    import torch
    return float(torch.stack([t.double().square().sum() for t in ts]).sum().sqrt())


def _clip_is_right(mr, ts, norm64, bound):
    """fp32 outputs: the norm's bound in the factor, the factor's rounding and the product's."""
    import torch
    norm, out = torch.zeros(1, device="cuda"), [torch.empty_like(t) for t in ts]
    mr.mr_clip_grad_norm(ts, out, norm64 / 3, norm=norm)
    for t, o in zip(ts, out):
        want = t.double() / 3
        assert bool(((o.double() - want).abs() <= (bound / norm64 + 3 * U) * 1.01 * want.abs()).all())
    return float(norm)


SIZES = [1, 2, 7, 31, 64, 1000, 4097, 50001, 262144, 300003, 1000003, 3000001, 5000000, 8000009, 12345678, 20000003]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("power", [0, 100, -100])
@pytest.mark.parametrize("offset", [0, 1])
def test_exact_pairs(mr, dtype, power, offset):
    """bf16 values from 1/4 to 4, times a power of 2: their squares are whole
    multiples of 2^-18 below 16, two of them fit 24 bits.  The sum in 64 bits is
    exact too.  The norm is the nearest fp32 value or a tie's neighbour."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(power + offset)
    for n in SIZES:
        x = torch.exp2(torch.rand(n + offset, generator=g, device="cuda") * 3.99 - 2).bfloat16()[offset:].double().clamp(max=3.984375)
        x *= torch.where(torch.rand(n, generator=g, device="cuda") < 0.5, -1.0, 1.0)
        raw = torch.empty(n + offset, dtype=torch.float32 if dtype == "fp32" else torch.bfloat16, device="cuda")
        t = raw[offset:]
        t.copy_(x * 2.0 ** power)
        want = _norm64([x]) * 2.0 ** power
        norm = torch.zeros(1, device="cuda")
        mr.mr_grad_norm([t], norm)
        assert abs(float(norm) - want) <= _half_step(want) + 2.0 ** -36 * want, n
        if dtype == "fp32":
            assert _clip_is_right(mr, [t], want, _half_step(want) + 2.0 ** -36 * want) == float(norm)


@pytest.mark.parametrize("dtype,pairs", [("bf16", 0.5 * U), ("fp32", U)])
def test_many_normal_values(mr, dtype, pairs):
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    for n in SIZES:
        t = torch.randn(n, generator=g, device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32) * 2.0 ** -14
        norm = torch.zeros(1, device="cuda")
        mr.mr_grad_norm([t, t[: n // 3]], norm)
        want = _norm64([t, t[: n // 3]])
        assert abs(float(norm) - want) <= _half_step(want) + (pairs + 2.0 ** -36) * want, n


def test_large_and_small_tiles_together(mr):
    """Tensors whose squares lie beside fp32's range on either side, and within it, in one list."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(2)
    parts = [torch.randn(n, generator=g, device="cuda") for n in (70001, 33, 100000, 5, 40000)]
    for powers in ((-100, -90, -120, -80, -140), (0, -100, -40, 20, -29), (60, 63, 0, -100, 70), (100, 0, 110, 64, 20), (-30, -29, -31, -28, -33),
                   (-60, -29, -140, -30, -100), (40, 58, 62, 64, 61)):
        ts = [p * 2.0 ** e for p, e in zip(parts, powers)]
        norm = torch.zeros(1, device="cuda")
        mr.mr_grad_norm(ts, norm)
        want = _norm64(ts)
        assert abs(float(norm) - want) <= _half_step(want) + (U + 2.0 ** -36) * want, powers


def _list(count, each):
    import torch
    flat = torch.randn(count * each, generator=torch.Generator().manual_seed(count)).cuda()
    return [flat[i * each:i * each + each - i % 3] for i in range(count)]


@pytest.mark.parametrize("count", [1024, 1025, 1536, 40000])
def test_lists_of_many_launches(mr, count):
    """Parts that every CTA joins for itself, and parts that are joined before."""
    import torch
    ts = _list(count, 40)
    want = _norm64(ts)
    norm = torch.zeros(1, device="cuda")
    mr.mr_grad_norm(ts, norm)
    assert abs(float(norm) - want) <= _half_step(want) + (U + 2.0 ** -36) * want
    assert _clip_is_right(mr, ts, want, _half_step(want) + (U + 2.0 ** -36) * want) == float(norm)
    mr.mr_clip_grad_norm(ts, ts, want / 7)              # in place, the norm not asked for
    mr.mr_grad_norm(ts, norm)
    assert abs(float(norm) - want / 7) <= 8 * U * want / 7


def test_time_grows_with_the_list(mr):
    """16 times the tensors take about 16 times as long, not 53 times (2.92 against 0.055 ms,
    where every CTA of the clipping joined the whole list's sums)."""
    import torch
    best = []
    for count in (2048, 32768):
        ts = _list(count, 512)
        work = torch.empty(mr.mr_grad_norm_workspace_bytes(count), dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        mr.mr_clip_grad_norm(ts, ts, 1e9, workspace=work)
        with torch.cuda.graph(graph):
            mr.mr_clip_grad_norm(ts, ts, 1e9, workspace=work)
        times = []
        for _ in range(20):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            graph.replay()
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        best.append(min(times))
    assert best[1] < 32 * best[0], best
