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

ALIAS, CUDA = 3, 4
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
