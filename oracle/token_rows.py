"""Rows of a table by token and the gated feed-forward block in 64 bits, from their definitions, with the
absolute values that bound what rounding can do to them.  Plain numpy."""
from __future__ import annotations

import numpy as np


def embed(table, ids, scale):
    x = np.zeros((len(ids), table.shape[1]))
    for t, i in enumerate(ids):
        if 0 <= i < len(table):
            x[t] = scale * np.asarray(table[i], np.float64)
    return x


def embed_grad(dx, ids, vocab, scale):
    """(gradient, sum of the terms' magnitudes, number of terms of each row)"""
    g, mag, count = np.zeros((vocab, dx.shape[1])), np.zeros((vocab, dx.shape[1])), np.zeros(vocab, np.int64)
    for t, i in enumerate(ids):
        if 0 <= i < vocab:
            g[i] += scale * dx[t]
            mag[i] += abs(scale) * np.abs(dx[t])
            count[i] += 1
    return g, mag, count


def act(x, name):
    """act(x) and its derivative."""
    with np.errstate(over="ignore", invalid="ignore"):
        if name == "relu":
            return np.where(x < 0, 0.0, x), (x > 0).astype(np.float64)
        if name == "silu":
            s = 1 / (1 + np.exp(-x))
            return x * s, s + x * s * (1 - s)
        z = np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3)
        t = np.tanh(z)
        return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * np.sqrt(2 / np.pi) * (1 + 3 * 0.044715 * x * x)


def feed_forward(x, wg, wu, wd, name, unit, half, tiny):
    """gate, up, h, y of one block, each with a bound of the error of sums in 32 bits (each term's
    rounding `unit`, as many as there are terms) and roundings to the type (`half` of the value, `tiny`
    where it is subnormal), h rounded."""
    d, f = x.shape[1], wg.shape[0]
    g, u = x @ wg.T, x @ wu.T
    eg, eu = d * unit * (np.abs(x) @ np.abs(wg).T), d * unit * (np.abs(x) @ np.abs(wu).T)
    a, _ = act(g, name)
    h = a * u
    ea = 1.2 * eg + 2.0 ** -19 * (np.abs(a) + np.abs(g) * 1e-3)  # slopes lie below 1.2; 2^x and the quotient
    eh = ea * np.abs(u) + np.abs(a) * eu + ea * eu
    eh = eh + half * (np.abs(h) + eh) + tiny
    y = h @ wd.T
    ey = eh @ np.abs(wd).T + f * unit * ((np.abs(h) + eh) @ np.abs(wd).T)
    return {"gate": (g, eg + half * np.abs(g) + tiny), "up": (u, eu + half * np.abs(u) + tiny),
            "y": (y, ey + half * (np.abs(y) + ey) + tiny)}


def feed_forward_grad(x, wg, wu, wd, name, gate, up, dy, unit, half, tiny):
    """dx, dwg, dwu, dwd from the gate and up given, with bounds as above."""
    rows, d, f = x.shape[0], x.shape[1], wg.shape[0]
    a, slope = act(gate, name)
    e_act = 2.0 ** -19 * np.abs(a) + 1e-6 * np.abs(gate) * 1e-2
    e_slope = 2.0 ** -17 if name != "relu" else 0.0

    def rounded(v, e):
        return v, e + half * (np.abs(v) + e) + tiny

    dh = dy @ wd
    edh = d * unit * (np.abs(dy) @ np.abs(wd)) + 4 * unit * np.abs(dh)
    dg, edg = rounded(dh * up * slope, edh * np.abs(up * slope) + (np.abs(dh) + edh) * np.abs(up) * e_slope)
    du, edu = rounded(dh * a, edh * np.abs(a) + (np.abs(dh) + edh) * e_act)
    h, eh = rounded(a * up, e_act * np.abs(up))

    def product(pairs, terms):
        v = sum(p @ q for (p, _), (q, _) in pairs)
        e = sum(ep @ np.abs(q) + np.abs(p) @ eq + ep @ eq + terms * unit * ((np.abs(p) + ep) @ (np.abs(q) + eq))
                for (p, ep), (q, eq) in pairs)
        return rounded(v, e)

    def sure(m):
        return m, np.zeros_like(m)

    def t(pair):
        return pair[0].T, pair[1].T

    return {"dx": product([((dg, edg), sure(wg)), ((du, edu), sure(wu))], 2 * f),
            "dw_gate": product([(t((dg, edg)), sure(x))], rows),
            "dw_up": product([(t((du, edu)), sure(x))], rows),
            "dw_down": product([(sure(dy.T), (h, eh))], rows)}
