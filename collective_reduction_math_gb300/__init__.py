"""Python binding of libmr.so, the C-ABI library of collective reduction math
on one GPU (see include/mr.h for the contract).

Argument marshalling only: every step of every collective runs in the CUDA
kernels of libmr.so.  PyTorch supplies the device memory and the stream.  If
the library has not been built, every call raises instead of computing
anything elsewhere.

    import torch, collective_reduction_math_gb300 as mr
    xs = [torch.randn(1 << 20, device="cuda") for _ in range(8)]
    ys = [torch.empty_like(x) for x in xs]
    mr.mr_allreduce(xs, ys, op="avg", algo="ring")
"""
from __future__ import annotations

import array
import ctypes
import os
import threading

__all__ = [
    "mr_allreduce", "mr_reduce_scatter", "mr_all_gather", "mr_allreduce_ex", "mr_reduce_scatter_ex", "mr_allreduce_rmsnorm", "mr_allreduce_sign_ef",
    "mr_reduce_scatter_sign_ef", "mr_reduce_scatter_sign_ef_noalloc", "mr_sign_ef_workspace_bytes",
    "mr_logprob", "mr_logprob_grad", "mr_distill_topk", "mr_distill_topk_grad", "mr_distill_topk_step",
    "mr_embedding", "mr_embedding_grad", "mr_embedding_grad_workspace_bytes", "mr_adjust_logits", "mr_adjust_logits_grad",
    "mr_grad_norm", "mr_clip_grad_norm", "mr_grad_norm_workspace_bytes",
    "mr_status_string", "mr_last_error",
    "mr_allreduce_ptrs", "mr_plan_auto", "mr_plan_ring_order", "mr_plan_tree", "mr_chunk_lo", "mr_launch_count", "mr_launch_floor", "MRError",
    "load", "LIB_PATH",
    "DTYPES", "OPS", "ALGOS", "DISTILL_MODES", "MAX_RANKS", "MAX_TOP", "MAX_TEACHER", "MAX_BIAS",
    "MAX_EMBEDDING_GRAD_ROWS",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmr.so")
MAX_RANKS = 64
MAX_TOP = 64            # top alternatives per row of mr_logprob
MAX_TEACHER = 128       # teacher entries per row of mr_distill_topk
MAX_BIAS = 1024         # biases per row of mr_adjust_logits
MAX_EMBEDDING_GRAD_ROWS = 262144    # rows of a call of mr_embedding_grad
DTYPES = {"fp32": 0, "bf16": 1, "int32": 2}
OPS = {"sum": 0, "prod": 1, "min": 2, "max": 3, "avg": 4}
ALGOS = {"ring": 0, "tree": 1, "hier": 2, "auto": 3}
DISTILL_MODES = {"renorm": 0, "tail": 1}
STATUS = {0: "MR_OK", 1: "MR_ERR_INVALID_ARGUMENT", 2: "MR_ERR_UNSUPPORTED", 3: "MR_ERR_ALIAS", 4: "MR_ERR_CUDA"}

_lib = None


class Order(ctypes.Structure):
    """mr_order_t: accumulation order for mr_allreduce_ex / mr_reduce_scatter_ex."""
    _fields_ = [("algo", ctypes.c_int), ("group", ctypes.c_int), ("per_hop_rounding", ctypes.c_int)]


class Adjust(ctypes.Structure):
    """mr_adjust_t: what mr_adjust_logits and its gradient do to each row."""
    _fields_ = [("history", ctypes.c_void_p), ("history_len", ctypes.c_size_t), ("n_history", ctypes.c_void_p),
                ("n_prompt", ctypes.c_void_p), ("repetition", ctypes.c_void_p), ("frequency", ctypes.c_void_p),
                ("presence", ctypes.c_void_p), ("bias_ids", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("bias_count", ctypes.c_int), ("mask", ctypes.c_void_p), ("ld_mask", ctypes.c_size_t)]


class MRError(RuntimeError):
    """A non-OK status from the library; ``status`` holds the code."""

    def __init__(self, status: int, detail: str):
        super().__init__(f"{STATUS.get(status, status)}: {detail}")
        self.status = status


def load():
    """Load libmr.so (built by ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build() first "
                           "(there is no fallback: the collectives run only in its CUDA kernels)")
    L = ctypes.CDLL(LIB_PATH)
    vp, sz, i = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    L.mr_allreduce.argtypes = [vp, vp, i, sz, i, i, i, vp]
    L.mr_allreduce.restype = i
    L.mr_reduce_scatter.argtypes = [vp, vp, i, sz, i, i, i, vp]
    L.mr_reduce_scatter.restype = i
    L.mr_all_gather.argtypes = [vp, vp, i, sz, i, vp]
    L.mr_all_gather.restype = i
    L.mr_allreduce_rmsnorm.argtypes = [vp, vp, i, sz, sz, vp, vp, vp, ctypes.c_float, i, i, vp]
    L.mr_allreduce_rmsnorm.restype = i
    L.mr_sign_ef_workspace_bytes.argtypes = [i, sz]
    L.mr_sign_ef_workspace_bytes.restype = sz
    for f in (L.mr_allreduce_sign_ef, L.mr_reduce_scatter_sign_ef):
        f.argtypes = [vp, vp, vp, vp, i, sz, i, i, vp, sz, vp]
        f.restype = i
    L.mr_reduce_scatter_sign_ef_noalloc.argtypes = [vp, vp, vp, vp, i, sz, i, i, vp]
    L.mr_reduce_scatter_sign_ef_noalloc.restype = i
    for f in (L.mr_allreduce_ex, L.mr_reduce_scatter_ex):
        f.argtypes = [vp, vp, i, sz, i, i, ctypes.POINTER(Order), vp]
        f.restype = i
    L.mr_status_string.argtypes = [i]
    L.mr_status_string.restype = ctypes.c_char_p
    L.mr_last_error.argtypes = []
    L.mr_last_error.restype = ctypes.c_char_p
    L.mr_plan_ring_order.argtypes = [i, i, vp]
    L.mr_plan_ring_order.restype = i
    L.mr_plan_tree.argtypes = [i, i, vp, vp, vp]
    L.mr_plan_tree.restype = i
    L.mr_chunk_lo.argtypes = [i, sz, i]
    L.mr_chunk_lo.restype = sz
    L.mr_plan_auto.argtypes = [i, sz, i, i, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_double)]
    L.mr_plan_auto.restype = i
    L.mr_launch_count.argtypes = []
    L.mr_launch_count.restype = ctypes.c_ulonglong
    L.mr_launch_floor.argtypes = [ctypes.c_uint, vp]
    L.mr_launch_floor.restype = i
    f = ctypes.c_float
    scores = [vp, vp, i, sz, sz, i, f]                      # logits, ld, W, rows, vocab, dtype, scale
    teacher = [i, vp, vp, i, f]                             # K, ids, values, mode, scale
    L.mr_logprob.argtypes = scores + [vp, i, vp, vp, vp, vp, vp, vp]
    L.mr_logprob_grad.argtypes = scores + [vp, vp, vp, vp, vp, vp, vp, vp]
    L.mr_distill_topk.argtypes = scores + teacher + [vp, vp, vp]
    L.mr_distill_topk_grad.argtypes = scores + teacher + [vp, vp, vp, vp, vp]
    L.mr_distill_topk_step.argtypes = scores + teacher + [vp, vp, vp, vp, vp]
    for g in (L.mr_logprob, L.mr_logprob_grad, L.mr_distill_topk, L.mr_distill_topk_grad, L.mr_distill_topk_step):
        g.restype = i
    L.mr_embedding.argtypes = [vp, vp, i, sz, sz, i, f, vp, sz, vp, sz, vp]
    L.mr_embedding_grad_workspace_bytes.argtypes = [sz, sz, sz]
    L.mr_embedding_grad.argtypes = [vp, sz, i, vp, sz, f, vp, vp, i, sz, sz, i, i, vp, sz, vp]
    L.mr_adjust_logits.argtypes = [vp, vp, i, sz, sz, i, vp, vp, vp, vp]
    L.mr_adjust_logits_grad.argtypes = [vp, vp, i, sz, sz, i, vp, vp, vp, vp, vp, vp]
    L.mr_grad_norm_workspace_bytes.argtypes = [i]
    L.mr_grad_norm.argtypes = [vp, vp, vp, i, vp, vp, sz, vp]
    L.mr_clip_grad_norm.argtypes = [vp, vp, vp, vp, i, f, vp, vp, sz, vp]
    for g in (L.mr_embedding, L.mr_embedding_grad, L.mr_adjust_logits, L.mr_adjust_logits_grad, L.mr_grad_norm, L.mr_clip_grad_norm):
        g.restype = i
    L.mr_embedding_grad_workspace_bytes.restype = sz
    L.mr_grad_norm_workspace_bytes.restype = sz
    _lib = L
    return L


# --------------------------------------------------------------------------
# marshalling helpers
# --------------------------------------------------------------------------

def _dtype_code(t) -> int:
    _setup()
    if t.dtype not in _codes:
        raise TypeError(f"unsupported dtype {t.dtype}: fp32, bf16 or int32")
    return _codes[t.dtype]


def _pointers(tensors):
    return (ctypes.c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _check(tensors, name):
    if not tensors:
        raise ValueError(f"{name}: empty list of rank buffers")
    d = tensors[0].dtype
    for t in tensors:
        if not t.is_cuda or not t.is_contiguous() or t.dtype != d:
            raise ValueError(f"{name}: rank buffers must be contiguous CUDA tensors of one dtype")


def _raise(status: int):
    L = load()
    raise MRError(status, L.mr_last_error().decode())


def _code(table, key, what):
    if isinstance(key, int):
        return key
    if key not in table:
        raise ValueError(f"unknown {what} {key!r}")
    return table[key]


# --------------------------------------------------------------------------
# the collectives (same names as the C ABI)
# --------------------------------------------------------------------------

def mr_allreduce(send, recv, op="sum", algo="ring", stream=None):
    """All-reduce: every recv[j] receives the reduction of send[0..W-1].
    send, recv: lists of W CUDA tensors of N elements (recv may be send)."""
    _check(send, "send")
    _check(recv, "recv")
    L = load()
    st = L.mr_allreduce(_pointers(send), _pointers(recv), len(send), send[0].numel(), _dtype_code(send[0]),
                        _code(OPS, op, "op"), _code(ALGOS, algo, "algo"), _stream(stream))
    if st:
        _raise(st)


def mr_reduce_scatter(send, recv, op="sum", algo="ring", stream=None):
    """Reduce-scatter: recv[k] (N/W elements) receives chunk k of the reduction
    of send[0..W-1] (N elements each)."""
    _check(send, "send")
    _check(recv, "recv")
    L = load()
    st = L.mr_reduce_scatter(_pointers(send), _pointers(recv), len(send), send[0].numel(), _dtype_code(send[0]),
                             _code(OPS, op, "op"), _code(ALGOS, algo, "algo"), _stream(stream))
    if st:
        _raise(st)


def mr_all_gather(send, recv, stream=None):
    """All-gather: every recv[j] (N elements) receives the concatenation of the
    shards send[0..W-1] (N/W elements each)."""
    _check(send, "send")
    _check(recv, "recv")
    L = load()
    st = L.mr_all_gather(_pointers(send), _pointers(recv), len(send), recv[0].numel(), _dtype_code(recv[0]),
                         _stream(stream))
    if st:
        _raise(st)


def _order(algo, group, per_hop):
    return Order(_code(ALGOS, algo, "algo"), int(group or 0), 1 if per_hop else 0)


def mr_allreduce_ex(send, recv, op="sum", algo="ring", group=None, per_hop=False, stream=None):
    """All-reduce with a choice of order: algo 'hier' folds groups of
    ``group`` consecutive ranks first, then the group totals; ``per_hop``
    rounds a bf16 running total to bf16 after every combine."""
    _check(send, "send")
    _check(recv, "recv")
    L = load()
    o = _order(algo, group, per_hop)
    st = L.mr_allreduce_ex(_pointers(send), _pointers(recv), len(send), send[0].numel(), _dtype_code(send[0]),
                           _code(OPS, op, "op"), ctypes.byref(o), _stream(stream))
    if st:
        _raise(st)


def mr_reduce_scatter_ex(send, recv, op="sum", algo="ring", group=None, per_hop=False, stream=None):
    """Reduce-scatter with a choice of order (see mr_allreduce_ex)."""
    _check(send, "send")
    _check(recv, "recv")
    L = load()
    o = _order(algo, group, per_hop)
    st = L.mr_reduce_scatter_ex(_pointers(send), _pointers(recv), len(send), send[0].numel(), _dtype_code(send[0]),
                                _code(OPS, op, "op"), ctypes.byref(o), _stream(stream))
    if st:
        _raise(st)


def mr_allreduce_rmsnorm(send, recv, weight, residual=None, residual_out=None, eps=1e-6, algo="ring",
                         stream=None):
    """All-reduce (sum) of send[0..W-1], residual add, then RMSNorm of every
    row of ``weight.numel()`` elements scaled by ``weight``; every recv[j]
    receives the normalised rows and residual_out (if given) the pre-norm sum
    plus residual."""
    _check(send, "send")
    _check(recv, "recv")
    L = load()
    hidden = weight.numel()
    n = send[0].numel()
    if hidden == 0 or n % hidden:
        raise ValueError("the buffers must hold whole rows of weight.numel() elements")
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    st = L.mr_allreduce_rmsnorm(_pointers(send), _pointers(recv), len(send), n // hidden, hidden, ptr(residual),
                                ptr(residual_out), weight.data_ptr(), float(eps), _dtype_code(send[0]),
                                _code(ALGOS, algo, "algo"), _stream(stream))
    if st:
        _raise(st)


def mr_sign_ef_workspace_bytes(W: int, N: int) -> int:
    return int(load().mr_sign_ef_workspace_bytes(W, N))


def _sign_ef(fn, grad, err, recv, scales, workspace, op, algo, stream):
    import torch
    _check(grad, "grad")
    _check(err, "err")
    _check(recv, "recv")
    for t in grad + err + recv:
        if t.dtype != torch.float32:
            raise TypeError("sign compression takes fp32 buffers")
    W, N = len(grad), grad[0].numel()
    need = mr_sign_ef_workspace_bytes(W, N)
    if workspace is None:        # plumbing: torch provides the device memory
        workspace = torch.empty(need, dtype=torch.uint8, device=grad[0].device)
    st = fn(_pointers(grad), _pointers(err), _pointers(recv), None if scales is None else scales.data_ptr(), W, N,
            _code(OPS, op, "op"), _code(ALGOS, algo, "algo"), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _stream(stream))
    if st:
        _raise(st)


def mr_allreduce_sign_ef(grad, err, recv, scales=None, workspace=None, op="avg", algo="ring", stream=None):
    """1-bit sign compression with error feedback, then all-reduce: every
    recv[j] gets the reduction of sign(grad[r] + err[r]) * s_r; err[r] is
    updated in place; scales (W fp32, optional) receives s_r."""
    _sign_ef(load().mr_allreduce_sign_ef, grad, err, recv, scales, workspace, op, algo, stream)


def mr_reduce_scatter_sign_ef(grad, err, recv, scales=None, workspace=None, op="avg", algo="ring", stream=None):
    """As mr_allreduce_sign_ef, but recv[k] (N/W elements) gets chunk k."""
    _sign_ef(load().mr_reduce_scatter_sign_ef, grad, err, recv, scales, workspace, op, algo, stream)


def mr_reduce_scatter_sign_ef_noalloc(grad, err, recv, scales=None, op="avg", algo="ring", stream=None):
    """mr_reduce_scatter_sign_ef without a workspace argument: the library
    uses its own fixed 64 KiB scratch, for callers that cannot allocate device
    memory.  Concurrent calls race on that scratch."""
    _check(grad, "grad")
    _check(err, "err")
    _check(recv, "recv")
    st = load().mr_reduce_scatter_sign_ef_noalloc(
        _pointers(grad), _pointers(err), _pointers(recv), None if scales is None else scales.data_ptr(), len(grad),
        grad[0].numel(), _code(OPS, op, "op"), _code(ALGOS, algo, "algo"), _stream(stream))
    if st:
        _raise(st)


# --------------------------------------------------------------------------
# token scores over a vocabulary in shards
# --------------------------------------------------------------------------

def _score_rows(tensors, name):
    """W rank buffers [rows, columns of the rank] -> (pointers, strides, rows, vocab, dtype code)."""
    if not tensors:
        raise ValueError(f"{name}: empty list of rank buffers")
    W, t0 = len(tensors), tensors[0]
    rows, dtype = t0.shape[0], t0.dtype
    ptrs, lds, vocab = [], [], 0
    for r, t in enumerate(tensors):
        shape = t.shape
        if len(shape) != 2 or not t.is_cuda or t.dtype is not dtype or shape[0] != rows:
            raise ValueError(f"{name}: rank buffers must be 2-D CUDA tensors [rows, columns] of one dtype")
        n = shape[1]
        ld, step = t.stride()
        if (step != 1 and n > 1) or (ld < n and rows > 1):
            raise ValueError(f"{name}[{r}]: the columns of a row must lie beside each other and rows must not overlap")
        ptrs.append(t.data_ptr())
        lds.append(ld if ld > n else n)
        vocab += n
    if W > 1:
        for r, t in enumerate(tensors):
            if t.shape[1] != (r + 1) * vocab // W - r * vocab // W:
                raise ValueError(f"{name}[{r}]: {t.shape[1]} columns, but rank {r} of {W} holds columns "
                                 f"[{r * vocab // W}, {(r + 1) * vocab // W}) of {vocab}")
    return (ctypes.c_void_p * W)(*ptrs), (ctypes.c_size_t * W)(*lds), rows, vocab, _dtype_code(t0)


def _row_ptr(t, name, n, dtype):
    """The address of a per-row array of n elements (None stays None)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name}: a contiguous CUDA tensor of {dtype} with {n} elements is needed")
    return t.data_ptr()


def _score_stream(stream, t):
    """As _stream, by torch's direct lookup where it has one: these calls are short, and
    torch.cuda.current_stream() builds an object for each (3 us of a 12 us call on GB300's host)."""
    if stream is None:
        import torch
        direct = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if direct is not None:
            return direct(t.get_device())
    return _stream(stream)


def _grad_rows(logits, grad, rows, vocab, code):
    gp, gl, g_rows, g_vocab, g_code = _score_rows(grad, "grad")
    if len(grad) != len(logits) or g_rows != rows or g_vocab != vocab or g_code != code:
        raise ValueError("grad: rank buffers of the scores' shape and dtype are needed")
    return gp, gl


def mr_logprob(logits, ids=None, scale=1.0, logprob=None, entropy=None, stats=None, top_ids=None, top_logprob=None,
               stream=None):
    """Log probabilities of the given tokens, with entropy and top
    alternatives.  logits: W rank buffers [T, columns of the rank] (fp32 or
    bf16; rows may be strided); ids: [T] int64, negative leaves a row out.
    Outputs, each optional: logprob, entropy [T] fp32; stats [T, 2] fp32 (for
    mr_logprob_grad); top_ids [T, k] int64 and top_logprob [T, k] fp32.  y =
    scale * logits."""
    from torch import float32, int64
    xp, ld, rows, vocab, code = _score_rows(logits, "logits")
    k = top_ids.shape[-1] if top_ids is not None else top_logprob.shape[-1] if top_logprob is not None else 0
    st = load().mr_logprob(xp, ld, len(logits), rows, vocab, code, scale, _row_ptr(ids, "ids", rows, int64), k,
                           _row_ptr(logprob, "logprob", rows, float32), _row_ptr(entropy, "entropy", rows, float32),
                           _row_ptr(stats, "stats", 2 * rows, float32), _row_ptr(top_ids, "top_ids", k * rows, int64),
                           _row_ptr(top_logprob, "top_logprob", k * rows, float32), _score_stream(stream, logits[0]))
    if st:
        _raise(st)


def mr_logprob_grad(logits, ids, stats, grad, g_logprob=None, entropy=None, g_entropy=None, scale=1.0, stream=None):
    """Gradient of g_logprob . logprob + g_entropy . entropy with respect to
    the scores, into ``grad`` (W rank buffers; may be ``logits``).  stats and
    entropy are mr_logprob's outputs."""
    from torch import float32, int64
    xp, ld, rows, vocab, code = _score_rows(logits, "logits")
    gp, gl = _grad_rows(logits, grad, rows, vocab, code)
    st = load().mr_logprob_grad(xp, ld, len(logits), rows, vocab, code, scale, _row_ptr(ids, "ids", rows, int64),
                                _row_ptr(stats, "stats", 2 * rows, float32), _row_ptr(entropy, "entropy", rows, float32),
                                _row_ptr(g_logprob, "g_logprob", rows, float32),
                                _row_ptr(g_entropy, "g_entropy", rows, float32), gp, gl, _score_stream(stream, logits[0]))
    if st:
        _raise(st)


def _teacher(teacher_ids, teacher_val, rows, mode, teacher_scale):
    from torch import float32, int64
    if teacher_ids.dim() != 2:
        raise ValueError("teacher_ids: a [rows, K] tensor is needed")
    k = teacher_ids.shape[1]
    return (k, _row_ptr(teacher_ids, "teacher_ids", k * rows, int64), _row_ptr(teacher_val, "teacher_val", k * rows, float32),
            _code(DISTILL_MODES, mode, "mode"), teacher_scale)


def mr_distill_topk(logits, teacher_ids, teacher_val, loss=None, stats=None, mode="renorm", scale=1.0,
                    teacher_scale=1.0, stream=None):
    """Distillation loss [T] from a teacher's top entries (teacher_ids [T, K]
    int64, negative for no entry; teacher_val [T, K] fp32).  mode 'renorm'
    takes logits and renormalises them over the list, 'tail' takes log
    probabilities and treats the remaining mass as one more outcome.  stats
    [T, 4] is what mr_distill_topk_grad takes."""
    from torch import float32
    xp, ld, rows, vocab, code = _score_rows(logits, "logits")
    st = load().mr_distill_topk(xp, ld, len(logits), rows, vocab, code, scale,
                                *_teacher(teacher_ids, teacher_val, rows, mode, teacher_scale),
                                _row_ptr(loss, "loss", rows, float32), _row_ptr(stats, "stats", 4 * rows, float32),
                                _score_stream(stream, logits[0]))
    if st:
        _raise(st)


def mr_distill_topk_grad(logits, teacher_ids, teacher_val, stats, g_loss, grad, mode="renorm", scale=1.0,
                         teacher_scale=1.0, stream=None):
    """Gradient of g_loss . loss with respect to the scores, into ``grad`` (W
    rank buffers; may be ``logits``)."""
    from torch import float32
    xp, ld, rows, vocab, code = _score_rows(logits, "logits")
    gp, gl = _grad_rows(logits, grad, rows, vocab, code)
    st = load().mr_distill_topk_grad(xp, ld, len(logits), rows, vocab, code, scale,
                                     *_teacher(teacher_ids, teacher_val, rows, mode, teacher_scale),
                                     _row_ptr(stats, "stats", 4 * rows, float32), _row_ptr(g_loss, "g_loss", rows, float32),
                                     gp, gl, _score_stream(stream, logits[0]))
    if st:
        _raise(st)


def mr_distill_topk_step(logits, teacher_ids, teacher_val, weight, loss, grad, mode="renorm", scale=1.0,
                         teacher_scale=1.0, stream=None):
    """Loss [T] (unweighted; may be None) and the gradient of weight . loss in
    one kernel, which keeps a row on the chip between the two as far as it
    fits (``grad`` may be ``logits``)."""
    from torch import float32
    xp, ld, rows, vocab, code = _score_rows(logits, "logits")
    gp, gl = _grad_rows(logits, grad, rows, vocab, code)
    st = load().mr_distill_topk_step(xp, ld, len(logits), rows, vocab, code, scale,
                                     *_teacher(teacher_ids, teacher_val, rows, mode, teacher_scale),
                                     _row_ptr(weight, "weight", rows, float32), _row_ptr(loss, "loss", rows, float32), gp, gl,
                                     _score_stream(stream, logits[0]))
    if st:
        _raise(st)


# --------------------------------------------------------------------------
# embedding, adjusted scores, gradient norm
# --------------------------------------------------------------------------

# These calls are short (a single token's take 2 to 6 us of the GPU), and so is
# the way to them: torch is looked up once, a tensor is asked for what is needed
# and no more.
_torch = None
_current_device = None
_raw_stream = None
_codes = None       # of the dtypes


def _setup():
    """torch, and its ways to the current device and stream."""
    global _torch, _current_device, _raw_stream, _codes
    if _torch is None:
        import torch
        _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        _raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
                       or (lambda dev: torch.cuda.current_stream(dev).cuda_stream))
        _codes = {torch.float32: 0, torch.bfloat16: 1, torch.int32: 2}
        _torch = torch
    return _torch


def _on_device(dev, stream, fn, *args):
    """fn(*args, stream) with the tensors' device current; the current stream is that device's."""
    if _current_device() != dev:
        with _torch.cuda.device(dev):
            return _on_device(dev, stream, fn, *args)
    if stream is None:
        stream = _raw_stream(dev)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    st = fn(*args, stream)
    if st:
        _raise(st)


# Small workspaces are kept for the default stream, one for each host thread (a
# thread's calls on it run in order, it cannot be captured and does not end):
# torch's allocation took 7 of the 24 us of a short list's norm.
_KEPT_BYTES = 1 << 20
_kept = threading.local()


def _workspace(workspace, need, dev, stream):
    """(the caller's workspace, or one of torch's memory that belongs to the stream of the call; its address; its bytes)"""
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace: a contiguous CUDA tensor on the other tensors' device is needed")
        return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if stream is None and need <= _KEPT_BYTES and _raw_stream(dev) == 0:
        t = _kept.__dict__.get(dev)
        if t is None:
            t = _kept.__dict__[dev] = _torch.empty(_KEPT_BYTES, dtype=_torch.uint8, device=dev)
    elif stream is None:
        with _torch.cuda.device(dev):
            t = _torch.empty(need, dtype=_torch.uint8, device=dev)
    else:
        s = _torch.cuda.ExternalStream(stream, device=dev) if isinstance(stream, int) else stream
        with _torch.cuda.stream(s):
            t = _torch.empty(need, dtype=_torch.uint8, device=dev)
    return t, t.data_ptr(), need


def _at(a):
    """The address of an array's elements."""
    return a.buffer_info()[0]


def _rows_2d(t, name, dev):
    """(address, elements from a row to the next) of a 2-D CUDA tensor whose rows are dense."""
    if t.dim() != 2 or dev < 0 or t.get_device() != dev:
        raise ValueError(f"{name}: a 2-D CUDA tensor on the other tensors' device is needed")
    rows, n = t.shape
    ld, step = t.stride()
    if (step != 1 and n > 1) or (ld < n and rows > 1):
        raise ValueError(f"{name}: the elements of a row must lie beside each other and rows must not overlap")
    return t.data_ptr(), ld if ld > n else n


def _table(tensors, name):
    """W rank buffers [rows of the rank, hidden] -> (pointers, strides, vocab, hidden, dtype code, device)."""
    _setup()
    if not tensors:
        raise ValueError(f"{name}: empty list of rank buffers")
    W, t0 = len(tensors), tensors[0]
    dev, dtype, hidden, vocab = t0.get_device(), t0.dtype, t0.shape[-1], 0
    ptrs, lds, rows = (ctypes.c_void_p * W)(), (ctypes.c_size_t * W)(), []
    for r, t in enumerate(tensors):
        ptrs[r], lds[r] = _rows_2d(t, name, dev)
        if t.dtype is not dtype or t.shape[1] != hidden:
            raise ValueError(f"{name}: rank buffers must be of one dtype and row length")
        rows.append(t.shape[0])
    vocab = sum(rows)
    for r, n in enumerate(rows):
        if n != (r + 1) * vocab // W - r * vocab // W:
            raise ValueError(f"{name}[{r}]: {n} rows, but rank {r} of {W} holds rows "
                             f"[{r * vocab // W}, {(r + 1) * vocab // W}) of {vocab}")
    return ptrs, lds, vocab, hidden, _dtype_code(t0), dev


def _array(t, name, shape, dtype, dev):
    """The address of a contiguous array of that shape on that device (None stays None)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor of shape {tuple(shape)} on the other tensors' device is needed")
    return t.data_ptr()


def mr_embedding(table, ids, out, scale=1.0, stream=None):
    """out[t] = scale * table[ids[t]].  table: W rank buffers [rows of the
    rank, hidden] (fp32 or bf16; rows may be strided); ids: [T] int64, negative
    gives zeros, past the vocabulary NaN; out: [T, hidden] of the table's
    dtype."""
    tp, ld, vocab, hidden, code, dev = _table(table, "table")
    T = ids.numel()
    op, ld_out = _rows_2d(out, "out", dev)
    if out.dtype is not table[0].dtype or out.shape[0] != T or out.shape[1] != hidden:
        raise ValueError(f"out: [{T}, {hidden}] of the table's dtype is needed")
    _on_device(dev, stream, load().mr_embedding, tp, ld, len(table), vocab, hidden, code, scale,
               _array(ids, "ids", (T,), _torch.int64, dev), T, op, ld_out)


def mr_embedding_grad_workspace_bytes(rows: int, vocab: int, hidden: int) -> int:
    return int(load().mr_embedding_grad_workspace_bytes(rows, vocab, hidden))


def mr_embedding_grad(g_out, ids, grad, scale=1.0, accumulate=False, workspace=None, stream=None):
    """The gradient of mr_embedding: grad[v] (+)= scale * the sum of g_out[t]
    over the tokens with ids[t] == v.  g_out: [T, hidden] fp32 or bf16; grad: W
    rank buffers [rows of the rank, hidden], fp32 or bf16.  ``accumulate`` adds
    to what grad holds, else every row is written.  workspace:
    mr_embedding_grad_workspace_bytes(T, vocab, hidden) bytes (None: torch
    provides them)."""
    gp, ld_grad, vocab, hidden, code, dev = _table(grad, "grad")
    T = ids.numel()
    xp, ld_g = _rows_2d(g_out, "g_out", dev)
    if g_out.shape[0] != T or g_out.shape[1] != hidden:
        raise ValueError(f"g_out: [{T}, {hidden}] is needed")
    L = load()
    keep, ws, n = _workspace(workspace, L.mr_embedding_grad_workspace_bytes(T, vocab, hidden), dev, stream)
    _on_device(dev, stream, L.mr_embedding_grad, xp, ld_g, _dtype_code(g_out), _array(ids, "ids", (T,), _torch.int64, dev), T, scale, gp,
               ld_grad, len(grad), vocab, hidden, code, 1 if accumulate else 0, ws, n)


def _columns(tensors, name, like=None):
    """W rank buffers [rows, columns of the rank] -> (addresses, strides, widths, rows, dtype, device), the
    first two as arrays; `like`: the answer for the buffers that these have to be alike."""
    _setup()
    if not tensors:
        raise ValueError(f"{name}: empty list of rank buffers")
    t0 = tensors[0]
    dev, dtype, rows = t0.get_device(), t0.dtype, t0.shape[0]
    ptrs, lds, widths = array.array("Q"), array.array("Q"), []
    for t in tensors:
        shape = t.shape
        if len(shape) != 2 or dev < 0 or t.get_device() != dev or t.dtype is not dtype or shape[0] != rows:
            raise ValueError(f"{name}: rank buffers must be 2-D CUDA tensors [rows, columns] of one dtype on one device")
        n = shape[1]
        ld, step = t.stride()
        if (step != 1 and n > 1) or (ld < n and rows > 1):
            raise ValueError(f"{name}: the columns of a row must lie beside each other and rows must not overlap")
        ptrs.append(t.data_ptr())
        lds.append(ld if ld > n else n)
        widths.append(n)
    if like is None:
        W, vocab = len(tensors), sum(widths)
        for r, n in enumerate(widths):
            if n != (r + 1) * vocab // W - r * vocab // W:
                raise ValueError(f"{name}[{r}]: {n} columns, but rank {r} of {W} holds columns "
                                 f"[{r * vocab // W}, {(r + 1) * vocab // W}) of {vocab}")
    elif (widths, rows, dtype, dev) != like[2:]:
        raise ValueError(f"{name}: rank buffers of the scores' shape, dtype and device are needed")
    return ptrs, lds, widths, rows, dtype, dev


def _adjust(rows, vocab, dev, history, n_history, n_prompt, repetition, frequency, presence, bias_ids, bias, mask):
    int64, float32, each = _torch.int64, _torch.float32, (rows,)
    h = ids = values = m = None
    L = K = ld_mask = 0
    if history is not None:
        if history.dim() != 2:
            raise ValueError("history: a [rows, entries] tensor is needed")
        L = history.shape[1]
        h = _array(history, "history", (rows, L), int64, dev)
        n_history, n_prompt = _array(n_history, "n_history", each, int64, dev), _array(n_prompt, "n_prompt", each, int64, dev)
        repetition = _array(repetition, "repetition", each, float32, dev)
        frequency, presence = _array(frequency, "frequency", each, float32, dev), _array(presence, "presence", each, float32, dev)
        if L == 0:          # a history without entries is none
            h = n_history = n_prompt = repetition = frequency = presence = None
    elif not n_history is n_prompt is repetition is frequency is presence is None:
        raise ValueError("lengths and penalties need a history")
    if bias_ids is not None:
        if bias_ids.dim() != 2 or bias is None:
            raise ValueError("bias_ids: a [rows, entries] tensor is needed, and bias with it")
        K = bias_ids.shape[1]
        ids, values = _array(bias_ids, "bias_ids", (rows, K), int64, dev), _array(bias, "bias", (rows, K), float32, dev)
        if K == 0:
            ids = values = None
    elif bias is not None:
        raise ValueError("bias needs bias_ids")
    if mask is not None:
        if mask.dtype is not _torch.int32 or mask.dim() != 2 or mask.shape[0] != rows or mask.shape[1] * 32 < vocab:
            raise ValueError(f"mask: int32 words [{rows}, {(vocab + 31) // 32}] are needed")
        m, ld_mask = _rows_2d(mask, "mask", dev)
    return Adjust(h, L, n_history, n_prompt, repetition, frequency, presence, ids, values, K, m, ld_mask)


def mr_adjust_logits(logits, out, history=None, n_history=None, n_prompt=None, repetition=None, frequency=None, presence=None,
                     bias_ids=None, bias=None, mask=None, stream=None):
    """Scores with penalties for repeated tokens, biases, and a mask of the
    allowed tokens.  logits, out: W rank buffers [T, columns of the rank] (out
    may be logits).  history: [T, L] int64, of which row t has its first
    n_history[t] ([T] int64; None: L) entries, the first n_prompt[t] of them the
    prompt's; negative entries are none.  repetition (counts prompt and
    output), frequency and presence (output only): [T] fp32.  bias_ids [T, K]
    int64 and bias [T, K] fp32.  mask: [T, ceil(vocab / 32)] int32 words, bit c %
    32 of word c // 32 set where column c is allowed."""
    x = _columns(logits, "logits")
    o = _columns(out, "out", x)
    xp, ld, widths, rows, _, dev = x
    vocab = sum(widths)
    a = _adjust(rows, vocab, dev, history, n_history, n_prompt, repetition, frequency, presence, bias_ids, bias, mask)
    _on_device(dev, stream, load().mr_adjust_logits, _at(xp), _at(ld), len(logits), rows, vocab, _dtype_code(logits[0]),
               ctypes.addressof(a), _at(o[0]), _at(o[1]))


def mr_adjust_logits_grad(logits, g_out, grad, history=None, n_history=None, n_prompt=None, repetition=None, frequency=None,
                          presence=None, mask=None, stream=None):
    """The gradient of mr_adjust_logits with respect to the scores: grad (W
    rank buffers; may be ``g_out``, not ``logits``) from g_out.  logits are the
    scores as they were before; frequency, presence and biases do not change
    the gradient."""
    x = _columns(logits, "logits")
    i, g = _columns(g_out, "g_out", x), _columns(grad, "grad", x)
    xp, ld, widths, rows, _, dev = x
    vocab = sum(widths)
    a = _adjust(rows, vocab, dev, history, n_history, n_prompt, repetition, frequency, presence, None, None, mask)
    _on_device(dev, stream, load().mr_adjust_logits_grad, _at(xp), _at(ld), len(logits), rows, vocab, _dtype_code(logits[0]),
               ctypes.addressof(a), _at(i[0]), _at(i[1]), _at(g[0]), _at(g[1]))


def mr_grad_norm_workspace_bytes(count: int) -> int:
    return int(load().mr_grad_norm_workspace_bytes(count))


def _tensor_list(tensors, name):
    """Any number of dense tensors -> (addresses, sizes, dtype codes, device), as arrays."""
    T = _setup().Tensor
    devices = set(map(T.get_device, tensors))
    if len(devices) > 1 or -1 in devices or not all(map(T.is_contiguous, tensors)):
        raise ValueError(f"{name}: contiguous CUDA tensors on one device are needed")
    try:
        codes = array.array("i", [_codes[t.dtype] for t in tensors])
    except KeyError as e:
        raise TypeError(f"{name}: unsupported dtype {e.args[0]}: fp32 or bf16") from None
    return (array.array("Q", map(T.data_ptr, tensors)), array.array("Q", map(T.numel, tensors)), codes,
            devices.pop() if devices else -1)


def _norm_call(fn, dev, norm, count, workspace, stream, *args):
    if dev < 0:         # no tensor: the norm's device
        if norm is None or norm.get_device() < 0:
            raise ValueError("norm: a CUDA tensor is needed")
        dev = norm.get_device()
    if norm is not None and (norm.dtype is not _torch.float32 or norm.numel() != 1 or norm.get_device() != dev):
        raise ValueError("norm: one fp32 value on the gradients' device is needed")
    keep, ws, n = _workspace(workspace, load().mr_grad_norm_workspace_bytes(count), dev, stream)
    _on_device(dev, stream, fn, *args, None if norm is None else norm.data_ptr(), ws, n)


def mr_grad_norm(grads, norm, workspace=None, stream=None):
    """norm[0] (fp32) receives the L2 norm of all tensors of the list (fp32 or
    bf16, mixed as they come) taken together.  workspace:
    mr_grad_norm_workspace_bytes(len(grads)) bytes (None: torch provides
    them)."""
    ptrs, sizes, codes, dev = _tensor_list(grads, "grads")
    if norm is None:
        raise ValueError("norm: a CUDA tensor is needed")
    _norm_call(load().mr_grad_norm, dev, norm, len(grads), workspace, stream, _at(ptrs), _at(sizes), _at(codes), len(grads))


def mr_clip_grad_norm(grads, out, max_norm, norm=None, workspace=None, stream=None):
    """out[i] = grads[i] * min(1, max_norm / norm) with the norm of all tensors
    taken together, which ``norm`` (one fp32 value, may be None) receives.
    ``out`` may be ``grads``, in whole or in part."""
    if len(out) != len(grads):
        raise ValueError("out: one tensor for each gradient is needed")
    ptrs, sizes, codes, dev = _tensor_list(grads, "grads")
    outs = ptrs
    if out is not grads:
        outs, out_sizes, out_codes, out_dev = _tensor_list(out, "out")
        if out_sizes != sizes or out_codes != codes or out_dev != dev:
            raise ValueError("out: tensors of the gradients' sizes, dtypes and device are needed")
    if not grads and norm is None:
        return
    _norm_call(load().mr_clip_grad_norm, dev, norm, len(grads), workspace, stream, _at(ptrs), _at(outs), _at(sizes), _at(codes),
               len(grads), max_norm)


def mr_allreduce_ptrs(send_ptrs, recv_ptrs, N, dtype, op, algo, stream):
    """The raw form: integer device pointers, as the C ABI takes them.
    Returns the status code instead of raising."""
    L = load()
    s = (ctypes.c_void_p * len(send_ptrs))(*send_ptrs)
    r = (ctypes.c_void_p * len(recv_ptrs))(*recv_ptrs)
    return L.mr_allreduce(s, r, len(send_ptrs), N, _code(DTYPES, dtype, "dtype"), _code(OPS, op, "op"),
                          _code(ALGOS, algo, "algo"), stream)


def mr_status_string(status: int) -> str:
    return load().mr_status_string(status).decode()


def mr_last_error() -> str:
    return load().mr_last_error().decode()


def mr_plan_ring_order(W: int, k: int):
    out = (ctypes.c_int * W)()
    st = load().mr_plan_ring_order(W, k, out)
    if st:
        _raise(st)
    return list(out)


def mr_plan_tree(W: int, which: int):
    """Returns (root, parent[W], children[W])."""
    parent = (ctypes.c_int * W)()
    child = (ctypes.c_int * (2 * W))()
    root = ctypes.c_int()
    st = load().mr_plan_tree(W, which, parent, child, ctypes.byref(root))
    if st:
        _raise(st)
    kids = [[c for c in child[2 * r:2 * r + 2] if c >= 0] for r in range(W)]
    return root.value, list(parent), kids


def mr_plan_auto(W: int, N: int, dtype: str, reduce_scatter: bool = False):
    """The order MR_AUTO picks for a call, and the cost model's time (us)."""
    a = ctypes.c_int()
    t = ctypes.c_double()
    st = load().mr_plan_auto(W, N, _code(DTYPES, dtype, "dtype"), int(reduce_scatter), ctypes.byref(a), ctypes.byref(t))
    if st:
        _raise(st)
    return {0: "ring", 1: "tree"}[a.value], t.value


def mr_chunk_lo(W: int, N: int, k: int) -> int:
    return int(load().mr_chunk_lo(W, N, k))


def mr_launch_count() -> int:
    return int(load().mr_launch_count())


def mr_launch_floor(ctas: int = 1, stream=None):
    """One empty kernel of ``ctas`` CTAs on the stream (the launch floor)."""
    st = load().mr_launch_floor(ctas, _stream(stream))
    if st:
        _raise(st)
