"""Refusals of the token-score calls on the host: every bad argument returns a
status before anything touches the GPU."""
import ctypes
import os

import pytest


def _gpu_visible():
    import torch
    return torch.cuda.is_available() or os.path.exists("/dev/nvidia0")


# Fake device addresses that must never be dereferenced: only where no GPU is.
pytestmark = pytest.mark.skipif(_gpu_visible(), reason="host-only checks with fake device addresses")

INVALID, UNSUPPORTED, ALIAS, CUDA = 1, 2, 3, 4
T, V, W = 6, 1001, 3
B = 1 << 40


@pytest.fixture(scope="module")
def mr():
    import __graft_entry__
    __graft_entry__.build()
    import collective_reduction_math_gb300 as m
    m.load()
    return m


def _ptrs(v):
    return (ctypes.c_void_p * len(v))(*v)


def _lds(v):
    return None if v is None else (ctypes.c_size_t * len(v))(*v)


def _shards(base, W=W, T=T, V=V, b=4):
    out = []
    for r in range(W):
        out.append(base)
        base += T * ((r + 1) * V // W - r * V // W) * b
    return out


def _at(i):
    return B + (1 << 32) + i * (1 << 20)


BASE = dict(logits=_shards(B), ld=None, W=W, T=T, V=V, dtype=0, scale=1.0, ids=_at(0), k=0, logprob=_at(1), entropy=None,
            stats=None, top_ids=None, top_logprob=None, stats_in=_at(2), entropy_in=_at(3), g_lp=_at(4), g_h=None,
            grad=_shards(B + (1 << 34)), ldg=None, K=4, t_ids=_at(5), t_val=_at(6), mode=0, t_scale=1.0, loss=_at(7),
            weight=_at(8))


def _head(a):
    return (None if a["logits"] is None else _ptrs(a["logits"]), _lds(a["ld"]), a["W"], a["T"], a["V"], a["dtype"], a["scale"])


def _call(mr, what, **kw):
    assert set(kw) <= set(BASE)
    a = dict(BASE, **kw)
    L = mr.load()
    grad = (None if a["grad"] is None else _ptrs(a["grad"]), _lds(a["ldg"]))
    teach = (a["K"], a["t_ids"], a["t_val"], a["mode"], a["t_scale"])
    if what == "logprob":
        return L.mr_logprob(*_head(a), a["ids"], a["k"], a["logprob"], a["entropy"], a["stats"], a["top_ids"], a["top_logprob"], None)
    if what == "logprob_grad":
        return L.mr_logprob_grad(*_head(a), a["ids"], a["stats_in"], a["entropy_in"], a["g_lp"], a["g_h"], *grad, None)
    if what == "distill":
        return L.mr_distill_topk(*_head(a), *teach, a["loss"], a["stats"], None)
    if what == "distill_grad":
        return L.mr_distill_topk_grad(*_head(a), *teach, a["stats_in"], a["g_lp"], *grad, None)
    return L.mr_distill_topk_step(*_head(a), *teach, a["weight"], a["loss"], *grad, None)


CALLS = ("logprob", "logprob_grad", "distill", "distill_grad", "distill_step")
WITH_GRAD = ("logprob_grad", "distill_grad", "distill_step")
DISTILL = ("distill", "distill_grad", "distill_step")


@pytest.mark.parametrize("what", CALLS)
def test_good_arguments_reach_the_launch(mr, what):
    # no GPU here: everything passes the checks and the launch itself is refused
    assert _call(mr, what) == CUDA
    assert _call(mr, what, dtype=1) == CUDA
    assert _call(mr, what, T=0) == 0            # nothing to do


@pytest.mark.parametrize("what", CALLS)
def test_shapes_and_scores(mr, what):
    for kw in (dict(W=0), dict(W=65), dict(dtype=3), dict(logits=None), dict(V=0), dict(V=1 << 31), dict(T=(1 << 40) + 1),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(logits=BASE["logits"][:2] + [0]), dict(logits=BASE["logits"][:2] + [BASE["logits"][2] + 2]),
               dict(ld=[333, 334, 333]), dict(ld=[400, 400, 1 << 41]), dict(T=1 << 30, ld=[1 << 33] * 3)):
        assert _call(mr, what, **kw) == INVALID, kw
        assert mr.mr_last_error()
    assert _call(mr, what, dtype=2) == UNSUPPORTED


@pytest.mark.parametrize("what", WITH_GRAD)
def test_gradient_buffers(mr, what):
    for kw in (dict(grad=None), dict(grad=BASE["grad"][:2] + [0]), dict(grad=[BASE["grad"][0] + 1] + BASE["grad"][1:]),
               dict(ldg=[10, 400, 400])):
        assert _call(mr, what, **kw) == INVALID, kw
    # in place is allowed, with the scores' own stride only
    assert _call(mr, what, grad=BASE["logits"]) == CUDA
    spaced = [B + r * (1 << 24) for r in range(3)]
    assert _call(mr, what, logits=spaced, grad=spaced, ld=[500] * 3, ldg=[500] * 3) == CUDA
    assert _call(mr, what, logits=spaced, grad=spaced, ld=[500] * 3, ldg=[600] * 3) == ALIAS
    assert _call(mr, what, grad=[BASE["logits"][0] + 4] + BASE["grad"][1:]) == ALIAS
    assert _call(mr, what, grad=[BASE["grad"][0], BASE["grad"][0] + 40, BASE["grad"][2]]) == ALIAS
    assert _call(mr, what, grad=[BASE["logits"][1]] + BASE["grad"][1:]) == ALIAS


@pytest.mark.parametrize("what", CALLS)
def test_column_slices_of_one_buffer(mr, what):
    lo = [r * V // W for r in range(W)]
    ld = [V + 7] * W
    x, g = [B + 4 * c for c in lo], [B + (1 << 34) + 4 * c for c in lo]
    assert _call(mr, what, logits=x, ld=ld, grad=g, ldg=ld) == CUDA
    if what in WITH_GRAD:
        assert _call(mr, what, logits=x, ld=ld, grad=x, ldg=ld) == CUDA
        g2 = [g[0], g[1] - 4, g[2]]             # one column into its neighbour
        assert _call(mr, what, logits=x, ld=ld, grad=g2, ldg=ld) == ALIAS
        wrap = [g[0], g[1], g[2] + 4 * 8]       # the last shard's end past the row into the next row's first
        assert _call(mr, what, logits=x, ld=ld, grad=wrap, ldg=ld) == ALIAS


def test_logprob_outputs(mr):
    for kw in (dict(k=-1), dict(k=65, top_ids=_at(20)), dict(k=5), dict(top_ids=_at(20)), dict(logprob=None), dict(ids=None),
               dict(k=5, top_ids=_at(20) + 4), dict(k=5, top_logprob=_at(20) + 2), dict(ids=_at(0) + 4), dict(logprob=_at(1) + 1),
               dict(stats=_at(20) + 2), dict(entropy=_at(20) + 3)):
        assert _call(mr, "logprob", **kw) == INVALID, kw
    assert _call(mr, "logprob", V=5, logits=_shards(B, V=5), k=6, top_ids=_at(20)) == INVALID
    assert _call(mr, "logprob", V=1 << 23, logits=[B, B + (1 << 30), B + (2 << 30)], k=5, ids=_at(1 << 13), logprob=None,
                 top_ids=_at(1 << 14)) == UNSUPPORTED
    assert _call(mr, "logprob", k=5, top_ids=_at(20), top_logprob=_at(21), entropy=_at(22), stats=_at(23)) == CUDA
    assert _call(mr, "logprob", k=5, top_ids=_at(20), logprob=None, ids=None) == CUDA
    for kw in (dict(logprob=_at(0)), dict(logprob=BASE["logits"][1]), dict(entropy=_at(1)), dict(stats=_at(1) + 8)):
        assert _call(mr, "logprob", **kw) == ALIAS, kw


def test_logprob_grad_arguments(mr):
    for kw in (dict(g_lp=None), dict(ids=None), dict(stats_in=None), dict(g_h=_at(9), entropy_in=None), dict(stats_in=_at(2) + 1),
               dict(g_lp=_at(4) + 2)):
        assert _call(mr, "logprob_grad", **kw) == INVALID, kw
    assert _call(mr, "logprob_grad", g_h=_at(9)) == CUDA
    assert _call(mr, "logprob_grad", g_h=_at(9), g_lp=None, ids=None) == CUDA
    assert _call(mr, "logprob_grad", stats_in=BASE["grad"][0]) == ALIAS


@pytest.mark.parametrize("what", DISTILL)
def test_teacher_arguments(mr, what):
    for kw in (dict(K=0), dict(K=129), dict(t_ids=None), dict(t_val=None), dict(t_ids=_at(5) + 4), dict(t_val=_at(6) + 2),
               dict(mode=2), dict(t_scale=0.0), dict(t_scale=float("nan")), dict(mode=1, t_scale=0.5)):
        assert _call(mr, what, **kw) == INVALID, kw
    assert _call(mr, what, mode=1) == CUDA
    if what == "distill":
        assert _call(mr, what, loss=None) == INVALID
        assert _call(mr, what, loss=None, stats=_at(20)) == CUDA
        assert _call(mr, what, loss=_at(5)) == ALIAS
    elif what == "distill_grad":
        assert _call(mr, what, stats_in=None) == INVALID
        assert _call(mr, what, g_lp=None) == INVALID
    else:
        assert _call(mr, what, weight=None) == INVALID
        assert _call(mr, what, loss=None) == CUDA
        assert _call(mr, what, loss=_at(8)) == ALIAS


def test_binding_refuses(mr):
    import torch
    x = [torch.zeros(4, 10)]
    with pytest.raises(ValueError, match="CUDA"):
        mr.mr_logprob(x, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="empty"):
        mr.mr_logprob([], None)
