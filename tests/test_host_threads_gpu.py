"""Host threads that call the library at the same time, each on a stream of its
own with sizes of its own, without the interpreter's lock between them
(tests/native/host_threads.c): no call is refused, and every result is that of
the call alone."""
import ctypes
import os
import shutil
import subprocess

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
ROUNDS, CALLS = 10, 200
TOP_K, STEP, NORM, GATHER = range(4)


class Job(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("W", ctypes.c_int), ("k", ctypes.c_int), ("last", ctypes.c_int), ("rows", ctypes.c_size_t),
                ("n", ctypes.c_size_t), ("ins", ctypes.c_void_p), ("outs", ctypes.c_void_p), ("a", ctypes.c_void_p), ("b", ctypes.c_void_p),
                ("c", ctypes.c_void_p), ("p", ctypes.c_void_p), ("q", ctypes.c_void_p), ("stream", ctypes.c_void_p),
                ("calls", ctypes.c_long), ("refused", ctypes.c_long)]


@pytest.fixture(scope="module")
def threads(tmp_path_factory):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("needs a C compiler")
    import __graft_entry__
    __graft_entry__.build()
    import collective_reduction_math_gb300 as mr
    mr.load()
    so = str(tmp_path_factory.mktemp("native") / "host_threads.so")
    subprocess.run([cc, "-O2", "-std=c11", "-pthread", "-shared", "-fPIC", "-I", os.path.join(os.path.dirname(HERE), "include"), "-o", so,
                    os.path.join(HERE, "native", "host_threads.c"), mr.LIB_PATH, "-Wl,-rpath," + os.path.dirname(mr.LIB_PATH)], check=True)
    return ctypes.CDLL(so)


def _random(rows, n, seed):
    import torch
    return torch.randn(rows, n, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)) * 2


class Call:
    """One thread's call: its buffers, and the structure that names them."""

    def __init__(self, kind, rows, n, ins, outs, k=0, a=None, b=None, c=None, p=None, q=None):
        import torch
        self.stream = torch.cuda.Stream()
        self.keep = (ins, outs, a, b, c, p, q)
        arrays = [(ctypes.c_void_p * max(1, len(t)))(*(x.data_ptr() for x in t)) for t in (ins, outs)]
        self.arrays, self.results = arrays, [t for t in list(outs) + [p, q] if t is not None]
        at = [None if t is None else t.data_ptr() for t in (a, b, c, p, q)]
        self.job = Job(kind, len(ins), k, 0, rows, n, ctypes.addressof(arrays[0]), ctypes.addressof(arrays[1]), *at,
                       self.stream.cuda_stream, 1, 0)


def _together(threads, calls):
    import torch
    torch.cuda.synchronize()
    want = []
    for c in calls:
        alone = (Job * 1)(c.job)
        assert threads.run_together(alone, 1) == 0 and alone[0].refused == 0, alone[0].last
        torch.cuda.synchronize()
        want.append([t.clone() for t in c.results])
        for t in c.results:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(ROUNDS):
        jobs = (Job * len(calls))(*(c.job for c in calls))
        for j in jobs:
            j.calls = CALLS
        assert threads.run_together(jobs, len(calls)) == 0
        torch.cuda.synchronize()
        assert [j.refused for j in jobs] == [0] * len(calls), [j.last for j in jobs]
    for c, first in zip(calls, want):
        for t, f in zip(c.results, first):
            assert torch.equal(t, f)


def test_steps_of_several_vocabularies(threads):
    import torch

    def call(V):
        T, K = 150, 8
        x = _random(T, V, V)
        ids = torch.arange(T * K, device="cuda").view(T, K)
        return Call(STEP, T, V, [x], [torch.empty_like(x)], K, ids, torch.zeros(T, K, device="cuda"), torch.ones(T, device="cuda"),
                    torch.empty(T, device="cuda"))

    # some 30 to 130 KB of a row in a CTA's shared memory
    _together(threads, [call(V) for V in (16384, 50257, 90000, 131072)])


def test_top_k_of_several_vocabularies(threads):
    import torch

    def call(V, k):
        T = 4
        return Call(TOP_K, T, V, [_random(T, V, V)], [], k, p=torch.empty(T, k, dtype=torch.int64, device="cuda"),
                    q=torch.empty(T, k, device="cuda"))

    _together(threads, [call(V, k) for V, k in ((262144, 64), (300007, 64), (400000, 64), (262144, 40))])


def test_norms_of_several_widths(threads):
    import torch

    def call(hidden):
        x = [_random(200, hidden, hidden + r) for r in range(2)]
        return Call(NORM, 200, hidden, x, [torch.empty_like(t) for t in x], a=torch.ones(hidden, device="cuda"))

    # rows of 64 to 192 KB of fp32
    _together(threads, [call(h) for h in (16384, 20480, 32768, 49152)])


def test_gathers_of_several_sizes(threads):
    import torch

    def call(n):
        return Call(GATHER, 0, 8 * n, [_random(1, n, n + r) for r in range(8)], [torch.empty(8 * n, device="cuda") for _ in range(8)])

    # one-wave grids of 2 to 4 CTAs an SM
    _together(threads, [call(n) for n in (262144, 393216, 524288, 589824)])
