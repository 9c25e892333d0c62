"""What the ends of a policy's step promise on the host: alias checks of the
most tensors that a call takes, and the sizes of workspaces."""
import ctypes
import os
import time

import pytest


def _gpu_visible():
    import torch
    return torch.cuda.is_available() or os.path.exists("/dev/nvidia0")


# Fake device addresses that must never be dereferenced: only where no GPU is.
no_gpu = pytest.mark.skipif(_gpu_visible(), reason="host-only checks with fake device addresses")

INVALID, ALIAS, CUDA = 1, 3, 4
B = 1 << 40


@pytest.fixture(scope="module")
def mr():
    import __graft_entry__
    __graft_entry__.build()
    import collective_reduction_math_gb300 as m
    m.load()
    return m


class Lists:
    """n tensors of 100 fp32 values each."""

    def __init__(self, mr, n):
        self.L, self.n, self.need = mr.load(), n, mr.mr_grad_norm_workspace_bytes(n)
        self.sizes, self.codes = (ctypes.c_size_t * n)(*([100] * n)), (ctypes.c_int * n)()

    def norm(self, at):
        return self.L.mr_grad_norm((ctypes.c_void_p * self.n)(*at), self.sizes, self.codes, self.n, B - 64, B + (1 << 36), self.need, None)

    def clip(self, at, out):
        return self.L.mr_clip_grad_norm((ctypes.c_void_p * self.n)(*at), (ctypes.c_void_p * self.n)(*out), self.sizes, self.codes, self.n, 1.0,
                                        B - 64, B + (1 << 36), self.need, None)


@no_gpu
def test_one_tensor_listed_many_times(mr):
    """The check is no slower than for as many tensors (65536 took 5 s where each met all others)."""
    n = 1 << 16
    lists, one, apart = Lists(mr, n), [B] * n, [B + 512 * i for i in range(n)]
    outs = [B + (1 << 32) + 512 * i for i in range(n)]
    start = time.perf_counter()
    assert lists.norm(apart) == CUDA and lists.norm(one) == CUDA
    assert lists.clip(apart, outs) == CUDA and lists.clip(one, outs) == CUDA
    assert lists.clip(apart, apart) == CUDA
    assert lists.norm([B + 4 * (i % 90) for i in range(n)]) == CUDA         # overlapping, all read
    # what is written meets each of them
    assert lists.clip(one, [B] + outs[1:]) == ALIAS
    assert lists.clip(apart, outs[:-1] + [apart[7] + 396]) == ALIAS
    assert lists.clip(apart, outs[:-1] + [outs[5] + 4]) == ALIAS
    assert lists.clip(apart, apart[1:] + apart[:1]) == ALIAS
    assert time.perf_counter() - start < 3.0


@no_gpu
def test_few_ranges_in_every_order(mr):
    """Three tensors and their outputs at all places of a short line: allowed exactly where
    each output is its own input or touches nothing."""
    lists, n = Lists(mr, 3), 400
    for a in range(0, 1200, 200):
        for o in range(0, 1600, 200):
            ins, outs = [B, B + a, B + 800], [B + (1 << 32), B + o, B + (1 << 33)]
            clear = all(abs(outs[1] - i) >= n for i in (ins[0], ins[2])) and (outs[1] == ins[1] or abs(outs[1] - ins[1]) >= n)
            assert lists.clip(ins, outs) == (CUDA if clear else ALIAS), (a, o)


def test_embedding_gradient_workspace(mr):
    need = mr.mr_embedding_grad_workspace_bytes
    assert need(0, 10, 10) > 0          # zeros are written: the sort's counts and the map of rows
    for few, many in (((0, 10, 10), (1, 10, 10)), ((31, 10, 10), (32, 10, 10)), ((1000, 50, 64), (1001, 50, 64)), ((4096, 50, 64), (262144, 50, 64)),
                      ((100, 10, 64), (100, 50000, 64)), ((100, 50000, 64), (100, (1 << 31) - 1, 64))):
        assert need(*few) <= need(*many)
    # a record and a token each, a bit a table row, and partial sums of rows with more than 32 tokens
    assert need(4096, 131072, 64) >= 4096 * 12 + 131072 // 8 + 2 * 128 * 64 * 4
    assert need(32, 10, 64) == need(32, 10, 4096)
    assert need(33, 10, 64) < need(33, 10, 4096)
    assert need(262144, 10, 64) > 0
    assert need(262145, 10, 64) == need(10, 1 << 31, 64) == need(10, 10, 1 << 31) == 0      # no such call


@no_gpu
@pytest.mark.parametrize("rows,hidden", [(0, 64), (6, 64), (40, 64), (262144, 8)])
def test_embedding_gradient_refuses_workspaces(mr, rows, hidden):
    V, L = 1001, mr.load()
    need = mr.mr_embedding_grad_workspace_bytes(rows, V, hidden)
    assert need > 0
    table, g, ids, ws = B, B + (1 << 36), B + (1 << 37), B + (1 << 38)

    def call(at=ws, size=need):
        return L.mr_embedding_grad(g, 0, 0, ids, rows, 1.0, (ctypes.c_void_p * 1)(table), None, 1, V, hidden, 0, 0, at, size, None)
    assert call() == CUDA
    for kw in (dict(at=None), dict(at=ws + 8), dict(size=need - 1), dict(size=0)):
        assert call(**kw) == INVALID, kw
    assert call(at=table + V * hidden * 4 - 16) == ALIAS
    if rows:
        assert call(at=g) == ALIAS and call(at=ids) == ALIAS
