"""Sparse rows: at most k entries in every row of a matrix that is made anew at each step.

    top = spmv.topk_rows(router_logits, k, weights="selected")     # a router's choice
    plan = spmv.RoutePlan(top.ids, experts, align=128)              # rows sorted by expert
    xs = plan.dispatch(x)                                           # tokens out ...
    y = plan.combine(ys, top.weights)                               # ... and back, weighted
    dys, dw = plan.combine_grad(dy, ys, top.weights)
    dx, dlogits = plan.dispatch_grad(dxs), top.grad(dw)

    t = spmv.topk_rows(teacher_logits, 64, lse=True)                # a teacher's top logits
    loss, dz = spmv.distill_loss_grad(z, t.ids, t.vals, teacher_lse=t.lse, scale=1 / len(z))

Every function takes CUDA tensors, enqueues on the current (or given) stream and returns
without waiting.  Results are allocated on that stream.  Gradients are functions of their
own; nothing is recorded by autograd.  They read the forward call's inputs and results again, where
no in-place change is noticed: a new tensor for scaled weights, no ``top.weights.mul_``.  The
semantics are those of ``include/spmv.h``.
"""
from __future__ import annotations

import contextlib
import functools

import torch

from ._abi import SPMV_BF16, SPMV_F16, SPMV_F32, WEIGHTINGS, _check, lib

_DTYPES = {torch.float32: SPMV_F32, torch.float16: SPMV_F16, torch.bfloat16: SPMV_BF16}
_F32, _I32, _empty = torch.float32, torch.int32, torch.empty

# the handle of a device's current stream, without the Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _current(t):
    """The current stream of a tensor's device (a host tensor is left for the library to refuse)."""
    device = t.get_device()
    return _raw_stream(device) if device >= 0 else None


@contextlib.contextmanager
def _on(stream, *inputs):
    """Make `stream` current for a call: results are allocated for it, and inputs of another
    stream are kept until it has read them."""
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    if stream != torch.cuda.current_stream():
        for t in inputs:
            if t is not None and t.is_cuda:
                t.record_stream(stream)
    with torch.cuda.stream(stream):
        yield


def _matrix(t, name, rows=None, cols=None, dtype=None):
    """(type code, leading dimension) of a row-major matrix of one of the row types."""
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, not {t.dtype}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    r, c = t.shape
    if (rows is not None and r != rows) or (cols is not None and c != cols):
        raise ValueError(f"{name} must be {rows if rows is not None else r} x {cols if cols is not None else c}, "
                         f"not {r} x {c}")
    s0, s1 = t.stride()
    if c > 1 and s1 != 1:
        raise ValueError(f"{name} must have unit column stride")
    if r > 1 and s0 < c:
        raise ValueError(f"{name} has overlapping rows")
    return code, (s0 if r > 1 else c)


def _plain(t, name, shape, dtype):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr() or None


def _out(t, name, like, rows, cols):
    """A new matrix of `like`'s type, or the checked one given, with its leading dimension."""
    if t is None:
        return _empty((rows, cols), dtype=like.dtype, device=like.device), cols
    return t, _matrix(t, name, rows, cols, like.dtype)[1]


class TopRows:
    """The k largest entries of every row of ``x``: ``ids`` (int32, -1 = none), and, where asked
    for, ``vals``, ``weights`` and ``lse`` (float32)."""

    __slots__ = ("ids", "vals", "weights", "lse", "_x", "_ids", "_weights", "_weighting", "_temperature")

    def grad(self, dweights, out=None, stream=None):
        """The gradient in x of a loss whose gradient in the weights is ``dweights``: the weights that
        topk_rows gave, whatever tensors the attributes have by then.  Neither they nor the ids may have been
        changed in place, nor, with weights over the row, x."""
        if stream is not None:
            with _on(stream, self._x, self._ids, self._weights, dweights, out):
                return self.grad(dweights, out)
        if not self._weighting:
            raise ValueError("topk_rows was called without weights")
        x, ids, weights = self._x, self._ids, self._weights
        rows, k = ids.shape
        n = x.shape[1]
        code, ldx = _matrix(x, "x")
        dw = _plain(dweights, "dweights", ids.shape, _F32)
        dx, lddx = _out(out, "out", x, rows, n)
        _check(lib.spmv_topk_rows_grad(rows, n, k, ids.data_ptr(), weights.data_ptr(), dw, self._weighting,
                                       self._temperature, x.data_ptr(), ldx, None, dx.data_ptr(), lddx, code,
                                       _current(x)))
        return dx


def topk_rows(x, k, temperature=1.0, weights=None, lse=False, vals=None, stream=None) -> TopRows:
    """The k largest entries of every row of x, values descending, ties to the lowest column;
    -inf is never taken (its id is -1).  ``weights``: None, "selected" (softmax over the
    chosen) or "row" (softmax over the row); ``lse``: also the row's log-sum-exp.  Both at
    ``temperature``.  ``vals``: whether the values themselves are wanted (None: unless weights
    are).  1 <= k <= min(n, 256)."""
    if stream is not None:
        with _on(stream, x):
            return topk_rows(x, k, temperature, weights, lse, vals)
    code, ldx = _matrix(x, "x")
    rows, n = x.shape
    weighting, k = WEIGHTINGS[weights], int(k)
    if not 1 <= k <= n or k > 256:
        raise ValueError("k must lie in [1, min(n, 256)]")
    top, device = TopRows(), x.device
    top._x, top._weighting, top._temperature = x, weighting, temperature
    top.ids = _empty((rows, k), dtype=_I32, device=device)
    top.vals = _empty((rows, k), dtype=_F32, device=device) if vals or (vals is None and not weighting) else None
    top.weights = _empty((rows, k), dtype=_F32, device=device) if weighting else None
    # (weights over the row come with it)
    top.lse = _empty((rows,), dtype=_F32, device=device) if lse or weighting == 2 else None
    _check(lib.spmv_topk_rows(rows, n, k, x.data_ptr(), ldx, code, temperature, weighting, top.ids.data_ptr(),
                              None if top.vals is None else top.vals.data_ptr(),
                              top.weights.data_ptr() if weighting else None,
                              None if top.lse is None else top.lse.data_ptr(), _current(x)))
    top._ids, top._weights = top.ids, top.weights
    return top


@functools.lru_cache(maxsize=4096)
def _plan_sizes(tokens, k, experts, align):
    """(rows of the sorted matrix, bytes of the plan's workspace)"""
    return (_check(lib.spmv_route_rows(tokens, k, experts, align)), _check(lib.spmv_route_workspace(tokens, k, experts)))


class RoutePlan:
    """Rows sorted by expert: the plan of one choice ``ids`` (int32, tokens x k; an entry
    outside [0, experts) is dropped).  ``rows`` is the sorted matrix's number of rows;
    ``offsets`` (experts + 1), ``slots`` (tokens x k) and ``sources`` (rows) as in spmv.h.
    Every call takes the tensors that these attributes have by then."""

    __slots__ = ("tokens", "k", "experts", "align", "rows", "offsets", "slots", "sources", "_known_slots",
                 "_known_sources")

    def __init__(self, ids, experts, align=1, stream=None):
        if stream is not None:
            with _on(stream, ids):
                return self.__init__(ids, experts, align)
        if ids.dim() != 2:
            raise ValueError("ids must be a matrix")
        ptr = _plain(ids, "ids", ids.shape, _I32)
        self.tokens, self.k = tokens, k = ids.shape
        self.experts, self.align = experts, align = int(experts), int(align)
        self.rows, work = _plan_sizes(tokens, k, experts, align)
        device = ids.device
        self.offsets = _empty((experts + 1,), dtype=_I32, device=device)
        self.slots = self._known_slots = slots = _empty((tokens, k), dtype=_I32, device=device)
        self.sources = self._known_sources = sources = _empty((self.rows,), dtype=_I32, device=device)
        space = _empty((work,), dtype=torch.uint8, device=device) if work else None
        _check(lib.spmv_route_plan(tokens, k, experts, align, ptr, self.offsets.data_ptr(), slots.data_ptr(),
                                   sources.data_ptr(), space.data_ptr() if work else None, work, _current(ids)))

    def _check_tensors(self):
        """The tensors that slots and sources have by now, where they are not the last call's."""
        _plain(self.slots, "slots", (self.tokens, self.k), _I32)
        _plain(self.sources, "sources", (self.rows,), _I32)
        self._known_slots, self._known_sources = self.slots, self.sources

    def dispatch(self, x, out=None, stream=None):
        """The tokens' rows sorted by expert (rows x d); rows without a source are 0."""
        if stream is not None:
            with _on(stream, self.slots, self.sources, x, out):
                return self.dispatch(x, out)
        slots, sources = self.slots, self.sources
        if slots is not self._known_slots or sources is not self._known_sources:
            self._check_tensors()
        code, ldx = _matrix(x, "x", self.tokens)
        d = x.shape[1]
        xs, ldxs = _out(out, "out", x, self.rows, d)
        _check(lib.spmv_route_dispatch(self.tokens, self.k, self.rows, d, slots.data_ptr(), sources.data_ptr(),
                                       x.data_ptr(), ldx, xs.data_ptr(), ldxs, code, _current(x)))
        return xs

    def combine(self, ys, weights=None, out=None, stream=None):
        """y[t] = sum over j of weights[t, j] ys[slots[t, j]] (weights None: all 1)."""
        if stream is not None:
            with _on(stream, self.slots, ys, weights, out):
                return self.combine(ys, weights, out)
        slots = self.slots
        if slots is not self._known_slots:
            self._check_tensors()
        code, ldys = _matrix(ys, "ys", self.rows)
        d = ys.shape[1]
        w = None if weights is None else _plain(weights, "weights", (self.tokens, self.k), _F32)
        y, ldy = _out(out, "out", ys, self.tokens, d)
        _check(lib.spmv_route_combine(self.tokens, self.k, self.rows, d, slots.data_ptr(), w, ys.data_ptr(), ldys,
                                      y.data_ptr(), ldy, code, _current(ys)))
        return y

    def combine_grad(self, dy, ys, weights, out=None, stream=None):
        """(dys, dweights): the gradients of combine in ys and in the weights."""
        if stream is not None:
            with _on(stream, self.slots, self.sources, dy, ys, weights, out):
                return self.combine_grad(dy, ys, weights, out)
        slots, sources = self.slots, self.sources
        if slots is not self._known_slots or sources is not self._known_sources:
            self._check_tensors()
        code, lddy = _matrix(dy, "dy", self.tokens)
        d = dy.shape[1]
        ldys = _matrix(ys, "ys", self.rows, d, dy.dtype)[1]
        w = _plain(weights, "weights", (self.tokens, self.k), _F32)
        dys, lddys = _out(out, "out", dy, self.rows, d)
        dw = _empty((self.tokens, self.k), dtype=_F32, device=dy.device)
        _check(lib.spmv_route_combine_grad(self.tokens, self.k, self.rows, d, slots.data_ptr(), sources.data_ptr(), w,
                                           dy.data_ptr(), lddy, ys.data_ptr(), ldys, dys.data_ptr(), lddys,
                                           dw.data_ptr(), code, _current(dy)))
        return dys, dw

    def dispatch_grad(self, dxs, out=None, stream=None):
        """The gradient of dispatch: dx[t] = sum over j of dxs[slots[t, j]]."""
        return self.combine(dxs, None, out, stream)


class DistillLoss:
    """``loss`` (float32, one a row, neither averaged nor scaled) and what its gradient needs."""

    __slots__ = ("loss", "stats", "_args", "_stats")

    def grad(self, dloss=None, scale=1.0, out=None, stream=None):
        """scale * dloss[t] * d loss[t] / d z[t] (dloss float32, None = all 1).  ``out`` may be
        the logits themselves, which the gradient then replaces (it can be taken once).  Neither the
        call's inputs nor ``stats`` may have been changed in place."""
        z, ids, teacher, lse, temperature = self._args
        stats = self._stats
        if stream is not None:
            with _on(stream, z, ids, teacher, lse, stats, dloss, out):
                return self.grad(dloss, scale, out)
        code, ldz = _matrix(z, "z")
        rows, vocab = z.shape
        g = None if dloss is None else _plain(dloss, "dloss", (rows,), _F32)
        dz, lddz = _out(out, "out", z, rows, vocab)
        _check(lib.spmv_distill_grad(rows, vocab, ids.shape[1], z.data_ptr(), ldz, code, ids.data_ptr(),
                                     teacher.data_ptr(), _DTYPES[teacher.dtype],
                                     None if lse is None else lse.data_ptr(), temperature, stats.data_ptr(), scale,
                                     g, dz.data_ptr(), lddz, _current(z)))
        return dz


def _distill_args(z, ids, teacher, teacher_lse):
    code, ldz = _matrix(z, "z")
    rows = z.shape[0]
    shape = ids.shape
    if len(shape) != 2 or shape[0] != rows:
        raise ValueError(f"ids must be a matrix of {rows} rows")
    i = _plain(ids, "ids", shape, _I32)
    tcode = _DTYPES.get(teacher.dtype)
    if tcode is None:
        raise TypeError(f"teacher must be float32, float16 or bfloat16, not {teacher.dtype}")
    t = _plain(teacher, "teacher", shape, teacher.dtype)
    lse = None if teacher_lse is None else _plain(teacher_lse, "teacher_lse", (rows,), _F32)
    return code, ldz, i, t, tcode, lse


def distill_loss(z, ids, teacher, teacher_lse=None, temperature=1.0, stream=None) -> DistillLoss:
    """The loss of logits z (rows x vocab) against a teacher's top logits: columns ``ids``
    (int32, rows x k, -1 = none, a column at most once) with logits ``teacher``.  With
    ``teacher_lse`` (the teacher's log-sum-exp over the whole vocabulary at the same
    temperature) the other columns count as one more class; without it the teacher's
    distribution is the softmax over the given entries."""
    if stream is not None:
        with _on(stream, z, ids, teacher, teacher_lse):
            return distill_loss(z, ids, teacher, teacher_lse, temperature)
    code, ldz, i, t, tcode, lse = _distill_args(z, ids, teacher, teacher_lse)
    rows, vocab = z.shape
    res = DistillLoss()
    res._args = (z, ids, teacher, teacher_lse, temperature)
    res.loss = _empty((rows,), dtype=_F32, device=z.device)
    res.stats = _empty((rows, 4), dtype=_F32, device=z.device)
    _check(lib.spmv_distill_loss(rows, vocab, ids.shape[1], z.data_ptr(), ldz, code, i, t, tcode, lse, temperature,
                                 res.loss.data_ptr(), res.stats.data_ptr(), _current(z)))
    res._stats = res.stats
    return res


def distill_loss_grad(z, ids, teacher, teacher_lse=None, temperature=1.0, scale=1.0, row_scale=None, out=None,
                      stream=None):
    """(loss, dz): :func:`distill_loss` and its gradient scale * row_scale[t] * d loss[t] / d z[t],
    reading z once.  ``out`` may be z itself, which the gradient then replaces."""
    if stream is not None:
        with _on(stream, z, ids, teacher, teacher_lse, row_scale, out):
            return distill_loss_grad(z, ids, teacher, teacher_lse, temperature, scale, row_scale, out)
    code, ldz, i, t, tcode, lse = _distill_args(z, ids, teacher, teacher_lse)
    rows, vocab = z.shape
    g = None if row_scale is None else _plain(row_scale, "row_scale", (rows,), _F32)
    loss = _empty((rows,), dtype=_F32, device=z.device)
    dz, lddz = _out(out, "out", z, rows, vocab)
    _check(lib.spmv_distill_loss_grad(rows, vocab, ids.shape[1], z.data_ptr(), ldz, code, i, t, tcode, lse, temperature,
                                      loss.data_ptr(), scale, g, dz.data_ptr(), lddz, _current(z)))
    return loss, dz
