"""Sparse rows in 64 bits, from their definitions: the k largest entries of a row, rows sorted by
expert and back, distillation from a teacher's top logits.  Plain numpy, one row at a time."""
from __future__ import annotations

import numpy as np

NEG_INF = -np.inf


def lse(x):
    """log sum exp, -inf for nothing above -inf, +inf for a +inf, NaN for a NaN."""
    x = np.asarray(x, np.float64)
    m = x.max(initial=NEG_INF)
    return m if not np.isfinite(m) else m + np.log(np.exp(x - m).sum())


def topk_row(x, k):
    """(ids, vals): the k largest, descending, ties to the lowest column; -inf is never taken,
    a NaN is above +inf."""
    x = np.asarray(x, np.float64)
    rank = np.where(np.isnan(x), np.inf, x)
    order = sorted((i for i in range(len(x)) if x[i] != NEG_INF), key=lambda i: (not np.isnan(x[i]), -rank[i], i))[:k]
    ids = np.full(k, -1, np.int64)
    vals = np.full(k, NEG_INF)
    ids[:len(order)] = order
    vals[:len(order)] = x[order]
    return ids, vals


def shares(x, tau):
    """Softmax of x / tau, by differences to the maximum (a log-sum of values near 1e38 would absorb
    how many there are); 0 where nothing is above -inf."""
    x = np.asarray(x, np.float64)
    m = x.max(initial=NEG_INF)
    if m == NEG_INF:
        return np.zeros(len(x))
    with np.errstate(invalid="ignore"):  # of a row with +inf or a NaN: NaN
        e = np.exp((x - m) / tau)
    return e / e.sum()


def top_weights(x, ids, vals, weighting, tau):
    """Softmax weights of the chosen entries, over the chosen or over the row."""
    q = shares(vals, tau) if weighting == "selected" else shares(x, tau)[ids]
    return np.array([0.0 if i < 0 else p for i, p in zip(ids, q)])


def top_weights_grad(x, ids, weights, dweights, weighting, tau):
    """Gradient in x of <dweights, weights>, from the softmax's Jacobian, written out."""
    x = np.asarray(x, np.float64)
    dx = np.zeros(len(x))
    q = shares(x, tau)
    chosen = [j for j, i in enumerate(ids) if i >= 0]
    for j in chosen:  # d w_j / d x_i = w_j ([i = id_j] - p_i) / tau
        dx[ids[j]] += dweights[j] * weights[j] / tau
        if weighting == "selected":
            for i in chosen:
                dx[ids[i]] -= dweights[j] * weights[j] * weights[i] / tau
        else:
            dx -= dweights[j] * weights[j] * q / tau
    return dx


def route_plan(ids, experts, align, rows):
    """(offsets, slots, sources) of the stable sort by expert."""
    flat = np.asarray(ids).reshape(-1)
    offsets = np.zeros(experts + 1, np.int64)
    slots, sources = np.full(flat.size, -1, np.int64), np.full(rows, -1, np.int64)
    for e in range(experts):
        at = offsets[e]
        for i in np.flatnonzero(flat == e):
            slots[i], sources[at] = at, i
            at += 1
        offsets[e + 1] = offsets[e] + -(-(at - offsets[e]) // align) * align
    return offsets, slots.reshape(np.shape(ids)), sources


def combine(ys, slots, weights):
    y = np.zeros((slots.shape[0], ys.shape[1]))
    for t in range(slots.shape[0]):
        for j, s in enumerate(slots[t]):
            if s >= 0:
                y[t] += (1.0 if weights is None else float(weights[t, j])) * ys[s]
    return y


def dispatch(x, slots, rows):
    xs = np.zeros((rows, x.shape[1]))
    for t in range(slots.shape[0]):
        for s in slots[t]:
            if s >= 0:
                xs[s] = x[t]
    return xs


def combine_grad(dy, ys, slots, weights):
    """(dys, dweights)"""
    dys, dw = np.zeros_like(ys, dtype=np.float64), np.zeros(slots.shape)
    for t in range(slots.shape[0]):
        for j, s in enumerate(slots[t]):
            if s >= 0:
                dys[s] = float(weights[t, j]) * dy[t]
                dw[t, j] = np.dot(dy[t], ys[s])
    return dys, dw


def _target(z, ids, teacher, teacher_lse, tau):
    """(columns, p, log p, r, log of the mass of the other columns under exp(z / tau), Z); None
    where the row has no target."""
    z = np.asarray(z, np.float64) / tau
    have = [j for j, i in enumerate(ids) if 0 <= i < len(z)]
    cols = np.array([ids[j] for j in have], np.int64)
    t = np.asarray(teacher, np.float64)[have] / tau
    if not have or (teacher_lse is None and t.max() == NEG_INF):
        return None
    logp = t - (lse(t) if teacher_lse is None else float(teacher_lse))
    p = np.exp(logp)
    others = np.ones(len(z), bool)
    others[cols] = False
    rest = 0.0 if teacher_lse is None or not others.any() else max(0.0, 1.0 - p.sum())
    return z, cols, p, logp, rest, others, lse(z[others]), lse(z)


def distill_loss(z, ids, teacher, teacher_lse=None, tau=1.0):
    t = _target(z, ids, teacher, teacher_lse, tau)
    if t is None:
        return 0.0
    z, cols, p, logp, rest, _, lse_rest, norm = t
    loss = sum(p[j] * (logp[j] - z[c] + norm) for j, c in enumerate(cols) if p[j] > 0)
    if rest > 0:
        loss += rest * (np.log(rest) - lse_rest + norm)
    return float(loss)


def distill_grad(z, ids, teacher, teacher_lse=None, tau=1.0):
    """d loss / d z = (softmax(z / tau) - target) / tau, the rest spread over the other columns
    as the student spreads it."""
    t = _target(z, ids, teacher, teacher_lse, tau)
    if t is None:
        return np.zeros(len(z))
    z, cols, p, _, rest, others, lse_rest, norm = t
    g = np.exp(z - norm)
    if rest > 0 and lse_rest > NEG_INF:
        share = np.exp(z[others] - z[others].max())  # (lse_rest itself would absorb the count at -1e38)
        g[others] -= rest * share / share.sum()
    g[cols] -= p
    return g / tau
