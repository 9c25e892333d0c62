"""Refusals of the embedding, adjusted-score and gradient-norm calls on the
host: every bad argument returns a status before anything touches the GPU; and
the 64-bit definitions against differences."""
import ctypes
import os

import numpy as np
import pytest

import step_ref as ref


def _gpu_visible():
    import torch
    return torch.cuda.is_available() or os.path.exists("/dev/nvidia0")


# Fake device addresses that must never be dereferenced: only where no GPU is.
no_gpu = pytest.mark.skipif(_gpu_visible(), reason="host-only checks with fake device addresses")

INVALID, UNSUPPORTED, ALIAS, CUDA = 1, 2, 3, 4
B = 1 << 40
FAR = B + (1 << 36)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def mr():
    import __graft_entry__
    __graft_entry__.build()
    import collective_reduction_math_gb300 as m
    m.load()
    return m


def _at(i):
    return FAR + i * (1 << 24)


def _ptrs(v):
    return None if v is None else (ctypes.c_void_p * max(1, len(v)))(*v)


def _sizes(v):
    return None if v is None else (ctypes.c_size_t * max(1, len(v)))(*v)


def _codes(v):
    return None if v is None else (ctypes.c_int * max(1, len(v)))(*v)


def _chunks(base, V, W, per):
    """Addresses of W chunks of V things of `per` bytes, one behind the other."""
    return [base + r * V // W * per for r in range(W)]


# ---- embedding ----
T, V, H, W = 6, 1001, 64, 3
EMBED = dict(table=_chunks(B, V, W, H * 4), ld=None, W=W, V=V, H=H, dtype=0, scale=1.0, ids=_at(0), T=T, out=_at(1), ld_out=0,
             g=_at(2), ld_g=0, g_dtype=0, accumulate=0, ws=_at(3), ws_bytes=1 << 23)


def _embed(mr, what, **kw):
    assert set(kw) <= set(EMBED)
    a = dict(EMBED, **kw)
    L = mr.load()
    if what == "lookup":
        return L.mr_embedding(_ptrs(a["table"]), _sizes(a["ld"]), a["W"], a["V"], a["H"], a["dtype"], a["scale"], a["ids"], a["T"],
                              a["out"], a["ld_out"], None)
    return L.mr_embedding_grad(a["g"], a["ld_g"], a["g_dtype"], a["ids"], a["T"], a["scale"], _ptrs(a["table"]), _sizes(a["ld"]), a["W"],
                               a["V"], a["H"], a["dtype"], a["accumulate"], a["ws"], a["ws_bytes"], None)


@no_gpu
@pytest.mark.parametrize("what", ["lookup", "grad"])
def test_embedding_arguments(mr, what):
    assert _embed(mr, what) == CUDA         # no GPU here: everything passes the checks and the launch itself is refused
    assert _embed(mr, what, dtype=1) == CUDA
    for kw in (dict(W=0), dict(W=65), dict(dtype=3), dict(table=None), dict(V=0), dict(V=1 << 31), dict(H=0), dict(H=1 << 31),
               dict(T=1 << 31), dict(scale=NAN), dict(scale=INF), dict(ids=None), dict(ids=_at(0) + 4),
               dict(table=EMBED["table"][:2] + [0]), dict(table=EMBED["table"][:2] + [EMBED["table"][2] + 2]),
               dict(ld=[64, 63, 64]), dict(ld=[64, 64, 1 << 41]), dict(V=(1 << 31) - 1, W=1, table=[B], ld=[1 << 40])):
        assert _embed(mr, what, **kw) == INVALID, kw
        assert mr.mr_last_error()
    assert _embed(mr, what, dtype=2) == UNSUPPORTED
    # fewer rows than ranks: the rank without one may be NULL
    assert _embed(mr, what, V=2, table=[0, B, B + 4096]) == CUDA


@no_gpu
def test_lookup_arguments(mr):
    for kw in (dict(out=None), dict(out=_at(1) + 2), dict(ld_out=63), dict(ld_out=1 << 41)):
        assert _embed(mr, "lookup", **kw) == INVALID, kw
    assert _embed(mr, "lookup", T=0, ids=None, out=None) == 0
    for kw in (dict(out=_at(0)), dict(out=EMBED["table"][1]), dict(out=EMBED["table"][0] - 4)):
        assert _embed(mr, "lookup", **kw) == ALIAS, kw
    # rows of the output beside the table's, in one buffer
    assert _embed(mr, "lookup", W=1, table=[B], ld=[128], out=B + 64 * 4, ld_out=128) == CUDA
    assert _embed(mr, "lookup", W=1, table=[B], ld=[128], out=B + 63 * 4, ld_out=128) == ALIAS


@no_gpu
def test_embedding_gradient_arguments(mr):
    for kw in (dict(g=None), dict(g=_at(2) + 2), dict(ld_g=63), dict(g_dtype=3), dict(accumulate=2), dict(accumulate=-1)):
        assert _embed(mr, "grad", **kw) == INVALID, kw
    assert _embed(mr, "grad", g_dtype=2) == UNSUPPORTED
    assert _embed(mr, "grad", g_dtype=1, dtype=0) == CUDA and _embed(mr, "grad", g_dtype=0, dtype=1) == CUDA
    assert _embed(mr, "grad", T=0, ids=None, g=None, accumulate=1) == 0
    assert _embed(mr, "grad", T=0, ids=None, g=None) == CUDA        # zeros are written
    for kw in (dict(g=EMBED["table"][1]), dict(ids=EMBED["table"][2] + 8), dict(table=[B, B, B + (1 << 30)])):
        assert _embed(mr, "grad", **kw) == ALIAS, kw
    assert _embed(mr, "grad", T=(1 << 18) + 1, ws_bytes=1 << 60) == UNSUPPORTED
    need = mr.mr_embedding_grad_workspace_bytes(T, V, H)
    if need:
        for kw in (dict(ws=None), dict(ws=_at(3) + 8), dict(ws_bytes=need - 1)):
            assert _embed(mr, "grad", **kw) == INVALID, kw
        assert _embed(mr, "grad", ws_bytes=need) == CUDA
        for kw in (dict(ws=_at(2)), dict(ws=EMBED["table"][0])):
            assert _embed(mr, "grad", **kw) == ALIAS, kw


# ---- adjusted scores ----
AV, AW = 1001, 3
SHARDS = [B + r * (1 << 20) for r in range(AW)]
LD = [400] * AW
ADJUST = dict(logits=SHARDS, ld=LD, W=AW, T=T, V=AV, dtype=0, out=[p + (1 << 30) for p in SHARDS], ld_out=LD, g=[p + (2 << 30) for p in SHARDS],
              ld_g=LD, adjust=True, history=_at(0), L=9, n_history=_at(1), n_prompt=_at(2), repetition=_at(3), frequency=_at(4),
              presence=_at(5), bias_ids=_at(6), bias=_at(7), K=5, mask=_at(8), ld_mask=0)
NO_LISTS = dict(history=None, L=0, n_history=None, n_prompt=None, repetition=None, frequency=None, presence=None)


def _adjust(mr, what, **kw):
    assert set(kw) <= set(ADJUST)
    a = dict(ADJUST, **kw)
    L = mr.load()
    c = mr.Adjust(a["history"], a["L"], a["n_history"], a["n_prompt"], a["repetition"], a["frequency"], a["presence"], a["bias_ids"],
                  a["bias"], a["K"], a["mask"], a["ld_mask"])
    p = ctypes.byref(c) if a["adjust"] else None
    head = (_ptrs(a["logits"]), _sizes(a["ld"]), a["W"], a["T"], a["V"], a["dtype"], p)
    if what == "adjust":
        return L.mr_adjust_logits(*head, _ptrs(a["out"]), _sizes(a["ld_out"]), None)
    return L.mr_adjust_logits_grad(*head, _ptrs(a["g"]), _sizes(a["ld_g"]), _ptrs(a["out"]), _sizes(a["ld_out"]), None)


@no_gpu
@pytest.mark.parametrize("what", ["adjust", "grad"])
def test_adjust_arguments(mr, what):
    assert _adjust(mr, what) == CUDA
    assert _adjust(mr, what, dtype=1) == CUDA
    assert _adjust(mr, what, T=0) == 0
    assert _adjust(mr, what, mask=None, K=0, bias=None, bias_ids=None, **NO_LISTS) == CUDA
    for kw in (dict(W=0), dict(W=65), dict(dtype=3), dict(logits=None), dict(out=None), dict(adjust=False), dict(V=0), dict(V=1 << 31),
               dict(T=(1 << 36) + 1), dict(logits=SHARDS[:2] + [0]), dict(logits=SHARDS[:2] + [SHARDS[2] + 2]), dict(ld=[333, 333, 400]),
               dict(ld_out=[400, 333, 400]), dict(ld=[400, 400, 1 << 41]), dict(L=0), dict(history=None), dict(L=1 << 30),
               dict(NO_LISTS, repetition=_at(3)), dict(NO_LISTS, n_prompt=_at(2)), dict(K=-1), dict(K=1025), dict(K=0), dict(bias=None),
               dict(bias_ids=None), dict(ld_mask=31), dict(ld_mask=1 << 41), dict(history=_at(0) + 4), dict(n_history=_at(1) + 4),
               dict(n_prompt=_at(2) + 1), dict(repetition=_at(3) + 2), dict(frequency=_at(4) + 1), dict(presence=_at(5) + 2),
               dict(bias_ids=_at(6) + 4), dict(bias=_at(7) + 2), dict(mask=_at(8) + 2), dict(T=1 << 36, L=(1 << 30) - 1)):
        assert _adjust(mr, what, **kw) == INVALID, kw
        assert mr.mr_last_error()
    assert _adjust(mr, what, dtype=2) == UNSUPPORTED
    assert _adjust(mr, what, ld_mask=40) == CUDA


@no_gpu
def test_adjust_overlaps(mr):
    assert _adjust(mr, "adjust", out=SHARDS) == CUDA            # in place
    for kw in (dict(out=SHARDS, ld_out=[500] * AW), dict(out=[SHARDS[1], SHARDS[0], SHARDS[2]]), dict(out=[SHARDS[0] + 4] + ADJUST["out"][1:]),
               dict(out=[ADJUST["out"][0]] * 3), dict(out=[_at(0)] + ADJUST["out"][1:]), dict(out=[_at(8)] + ADJUST["out"][1:]),
               dict(out=[_at(3)] + ADJUST["out"][1:])):
        assert _adjust(mr, "adjust", **kw) == ALIAS, kw
    assert _adjust(mr, "grad", out=ADJUST["g"]) == CUDA         # in place of what came back
    assert _adjust(mr, "grad", out=SHARDS) == ALIAS             # the scores are still looked at
    assert _adjust(mr, "grad", out=SHARDS, repetition=None) == CUDA
    assert _adjust(mr, "grad", logits=None, repetition=None) == CUDA
    assert _adjust(mr, "grad", g=None) == INVALID
    cuts = [4 * (r * AV // AW) for r in range(AW)]
    one, two = [B + c for c in cuts], [B + (1 << 30) + c for c in cuts]
    ld = [AV + 3] * AW
    assert _adjust(mr, "adjust", logits=one, out=two, ld=ld, ld_out=ld) == CUDA          # column slices
    assert _adjust(mr, "adjust", logits=one, out=one, ld=ld, ld_out=ld) == CUDA
    assert _adjust(mr, "adjust", logits=one, out=[two[0], two[1] - 4, two[2]], ld=ld, ld_out=ld) == ALIAS


# ---- gradient norm ----
TENSORS = dict(grad=[_at(0), _at(1), _at(2)], out=[_at(10), _at(11), _at(12)], n=[100, 0, 77], dtype=[0, 0, 1], count=3, max_norm=1.0, norm=_at(20),
               ws=_at(21), ws_bytes=1 << 20)


def _norm(mr, what, **kw):
    assert set(kw) <= set(TENSORS)
    a = dict(TENSORS, **kw)
    L = mr.load()
    if what == "norm":
        return L.mr_grad_norm(_ptrs(a["grad"]), _sizes(a["n"]), _codes(a["dtype"]), a["count"], a["norm"], a["ws"], a["ws_bytes"], None)
    return L.mr_clip_grad_norm(_ptrs(a["grad"]), _ptrs(a["out"]), _sizes(a["n"]), _codes(a["dtype"]), a["count"], a["max_norm"], a["norm"],
                               a["ws"], a["ws_bytes"], None)


@no_gpu
@pytest.mark.parametrize("what", ["norm", "clip"])
def test_norm_arguments(mr, what):
    assert _norm(mr, what) == CUDA
    assert _norm(mr, what, grad=[_at(0), 0, _at(2)], out=[_at(10), 0, _at(12)]) == CUDA         # nothing is there
    assert _norm(mr, what, count=0, grad=None, out=None, n=None, dtype=None) == CUDA           # a norm of 0
    for kw in (dict(count=-1), dict(count=(1 << 20) + 1), dict(grad=None), dict(n=None), dict(dtype=None), dict(dtype=[0, 0, 3]), dict(ws=None),
               dict(ws=_at(21) + 4), dict(ws_bytes=mr.mr_grad_norm_workspace_bytes(3) - 1), dict(norm=_at(20) + 2), dict(grad=[0, 0, _at(2)]),
               dict(grad=[_at(0) + 2, 0, _at(2)]), dict(grad=[_at(0), 0, _at(2) + 1]), dict(n=[100, 0, (1 << 40) + 1])):
        assert _norm(mr, what, **kw) == INVALID, kw
        assert mr.mr_last_error()
    assert _norm(mr, what, dtype=[0, 0, 2]) == UNSUPPORTED
    for kw in (dict(ws=_at(0)), dict(norm=_at(2)), dict(norm=_at(21))):
        assert _norm(mr, what, **kw) == ALIAS, kw
    assert _norm(mr, "norm", norm=None) == INVALID


@no_gpu
def test_clip_arguments(mr):
    for kw in (dict(max_norm=NAN), dict(max_norm=-1.0), dict(out=None), dict(out=[0, 0, _at(12)]), dict(out=[_at(10) + 1, 0, _at(12)])):
        assert _norm(mr, "clip", **kw) == INVALID, kw
    for kw in (dict(norm=None), dict(max_norm=0.0), dict(max_norm=INF), dict(out=TENSORS["grad"]), dict(out=[_at(0), 0, _at(12)])):
        assert _norm(mr, "clip", **kw) == CUDA, kw
    assert _norm(mr, "clip", count=0, grad=None, out=None, n=None, dtype=None, norm=None) == 0
    for kw in (dict(out=[_at(0) + 4, 0, _at(12)]), dict(out=[_at(2), 0, _at(12)]), dict(out=[_at(10), 0, _at(10) + 8]),
               dict(grad=[_at(0), 0, _at(0)], out=[_at(0), 0, _at(0)], dtype=[0, 0, 0])):
        assert _norm(mr, "clip", **kw) == ALIAS, kw
    assert _norm(mr, "norm", grad=[_at(0), 0, _at(0)]) == CUDA          # counted twice


def test_workspaces(mr):
    assert mr.mr_grad_norm_workspace_bytes(0) == mr.mr_grad_norm_workspace_bytes(512) > 0
    assert mr.mr_grad_norm_workspace_bytes(513) == 2 * mr.mr_grad_norm_workspace_bytes(512)
    assert mr.mr_embedding_grad_workspace_bytes(0, 10, 10) >= 0


def test_bindings_refuse(mr):
    import torch
    cpu = torch.zeros(4, 8)
    ids = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: mr.mr_embedding([cpu], ids, cpu), lambda: mr.mr_embedding([], ids, cpu), lambda: mr.mr_embedding_grad(cpu, ids, [cpu]),
                 lambda: mr.mr_adjust_logits([cpu], [cpu]), lambda: mr.mr_adjust_logits_grad([cpu], [cpu], [cpu]),
                 lambda: mr.mr_grad_norm([cpu], cpu), lambda: mr.mr_clip_grad_norm([cpu], [cpu], 1.0), lambda: mr.mr_grad_norm([], cpu),
                 lambda: mr.mr_clip_grad_norm([cpu], [], 1.0)):
        with pytest.raises(ValueError):
            call()


# ---- the definitions themselves ----

def test_definitions_against_differences():
    rng = np.random.default_rng(0)
    V, T, H = 9, 20, 3
    ids = rng.integers(-1, V + 1, T)
    g, table = rng.normal(size=(T, H)), rng.normal(size=(V, H))
    on = (ids >= 0) & (ids < V)
    value = lambda t: (g[on] * 0.7 * t[ids[on]]).sum()  # noqa: E731
    grad, _, _ = ref.embedding_grad(g, ids, V, 0.7, None)
    x = rng.normal(size=V) + 0.05
    x[np.abs(x) < 0.01] = 0.5
    history, allowed = rng.integers(-1, V, 6), rng.random(V) < 0.7
    row = lambda s: ref.adjusted_row(s, history, 2, 1.3, 0.2, 0.4, [1, 1, 4], [0.5, 0.25, -1.0], allowed)[0]  # noqa: E731
    back = ref.adjusted_grad_row(np.ones(V), x, history, 1.3, allowed)[0]
    h = 1e-6
    for v in range(V):
        for c in range(H):
            d = np.zeros_like(table)
            d[v, c] = h
            assert abs((value(table + d) - value(table - d)) / (2 * h) - grad[v, c]) < 1e-7
        d = np.zeros(V)
        d[v] = h
        got = (row(x + d)[v] - row(x - d)[v]) / (2 * h) if allowed[v] else 0.0
        assert abs(got - back[v]) < 1e-7
    assert abs(ref.norm([np.array([3e200, 0.0]), np.array([4e200])]) / 5e200 - 1) < 1e-15
