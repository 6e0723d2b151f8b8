"""Oracle of the operators around the layers: token embedding, norm of whole
rows, distillation from a teacher's top logits, forward and hand-derived
backward in fp64 (NumPy).
"""
from __future__ import annotations

import numpy as np

__all__ = ["embed", "embed_backward", "layer_norm", "layer_norm_backward", "distill"]


def embed(E, ids, scale=1.0):
    """Rows of E at the tokens; an id outside the vocabulary is no token."""
    E, ids = np.asarray(E, np.float64), np.asarray(ids)
    ok = (ids >= 0) & (ids < len(E))
    return np.where(ok[:, None], E[np.where(ok, ids, 0)] * scale, 0.0)


def embed_backward(ids, dY, vocab, scale=1.0):
    """The table's gradient, the sum of the magnitudes of its terms, and how
    many rows each id has."""
    ids, dY = np.asarray(ids), np.asarray(dY, np.float64)
    ok = (ids >= 0) & (ids < vocab)
    dE, mag = np.zeros((vocab, dY.shape[1])), np.zeros((vocab, dY.shape[1]))
    np.add.at(dE, ids[ok], dY[ok] * scale)
    np.add.at(mag, ids[ok], np.abs(dY[ok] * scale))
    return dE, mag, np.bincount(ids[ok], minlength=vocab)


def layer_norm(h, w, b=None, eps=1e-5, centered=True):
    """y, the normed rows u before the weight, and s."""
    h = np.asarray(h, np.float64)
    d = h - h.mean(-1, keepdims=True) if centered else h
    s = 1.0 / np.sqrt((d * d).mean(-1, keepdims=True) + eps)
    u = d * s
    y = u * np.asarray(w, np.float64)
    return (y if b is None else y + np.asarray(b, np.float64)), u, s


def layer_norm_backward(h, w, dy, dh=None, eps=1e-5, centered=True):
    """dx, dw, db and, for error bounds, the magnitudes of the terms of each (of
    those with u, u taken as |u| + 1: its error is relative to both)."""
    _, u, s = layer_norm(h, w, None, eps, centered)
    dy, w = np.asarray(dy, np.float64), np.asarray(w, np.float64)
    g = dy * w
    dx = g - u * (g * u).mean(-1, keepdims=True)
    if centered:
        dx = dx - g.mean(-1, keepdims=True)
    dx = dx * s
    a, v = np.abs(g), np.abs(u) + 1.0
    mx = s * (a + a.mean(-1, keepdims=True) + v * (a * v).mean(-1, keepdims=True))
    if dh is not None:
        dx, mx = dx + dh, mx + np.abs(dh)
    return dx, (dy * u).sum(0), dy.sum(0), mx, (np.abs(dy) * v).sum(0), np.abs(dy).sum(0)


def distill(z, top_ids=None, top_logits=None, labels=None, temperature=1.0, hard=0.0, with_loss=None, dloss=None):
    """Rows' losses and dz, and the magnitudes that their errors are relative to
    in steps of the arithmetic: ``n`` for each of a sum's terms, 1 for the rest.
    Returns (loss, dz, bound_loss(n), bound_dz(n))."""
    z = np.asarray(z, np.float64)
    T, V = z.shape
    rows = np.ones(T, bool) if with_loss is None else np.asarray(with_loss, bool)
    g = np.ones(T) if dloss is None else np.asarray(dloss, np.float64)
    tau = float(temperature)
    loss, dz = np.zeros(T), np.zeros((T, V))
    parts = []
    for t in np.nonzero(rows)[0]:
        x = z[t] - z[t].max()
        ones, many = 0.0, 0.0                            # a bound is ones + n many
        zones, zmany = np.zeros(V), np.zeros(V)
        if hard < 1.0:
            i, l = np.asarray(top_ids[t]), np.asarray(top_logits[t], np.float64)
            ok = (i >= 0) & (i < V) & (l > -np.inf)
            i, l = i[ok], l[ok] / tau
            if len(i):
                l = l - l.max()
                lp = l - np.log(np.exp(l).sum())
                p = np.exp(lp)
                e = np.exp(x / tau)
                lq = x[i] / tau - np.log(e.sum())
                q = e / e.sum()
                c = (1.0 - hard) * tau
                with np.errstate(invalid="ignore"):
                    loss[t] += c * tau * np.where(p > 0, p * (lp - lq), 0.0).sum()
                    size = np.where(p > 0, p * (np.abs(lp) + np.abs(lq) + np.abs(l) + np.abs(x[i]) / tau + 1), 0.0).sum()
                d = q.copy()
                np.add.at(d, i, -p)
                dz[t] += g[t] * c * d
                # an exponent: its difference, product and scale are rounded, 6 half steps of it
                far = np.where(q > 0, np.abs(np.where(q > 0, x, 0.0)) / tau, 0.0)
                near = 6 * (q * far).sum()
                tp = np.zeros(V)
                np.add.at(tp, i, p * (6 * np.abs(l) + 6 * (p * np.abs(l)).sum() + 8))
                tn = np.zeros(V)
                np.add.at(tn, i, p)
                zones += abs(g[t]) * c * (q * (6 * far + near + 8) + tp)
                zmany += abs(g[t]) * c * (q + tn)
                ones, many = ones + c * tau * (8 * size + near), many + c * tau * (1.0 + size)
        if hard > 0.0 and 0 <= labels[t] < V:
            e = np.exp(x)
            o = e / e.sum()
            ce = np.log(e.sum()) - x[labels[t]]
            loss[t] += hard * ce
            d = o.copy()
            d[labels[t]] -= 1.0
            dz[t] += g[t] * hard * d
            far = np.where(o > 0, np.abs(np.where(o > 0, x, 0.0)), 0.0)
            near = 6 * (o * far).sum()
            ones += hard * (4 * (abs(x[labels[t]]) + abs(np.log(e.sum())) + 1) + near)
            many += hard
            hit = np.zeros(V)
            hit[labels[t]] = 1.0
            zones += abs(g[t]) * hard * (o * (6 * far + near + 8) + 4 * hit)
            zmany += abs(g[t]) * hard * o
        parts.append((t, ones, many, zones, zmany))

    def bound_loss(n):
        b = np.zeros(T)
        for t, ones, many, _, _ in parts:
            b[t] = ones + n * many
        return b

    def bound_dz(n):
        b = np.zeros((T, V))
        for t, _, _, ones, many in parts:
            b[t] = ones + n * many
        return b
    return loss, dz, bound_loss, bound_dz
