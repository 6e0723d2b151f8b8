"""Oracle of the operators between the q/k/v and the o projection: rotary
positions, per-head norms, differential attention, forward and hand-derived
backward in fp64 (NumPy).  Tokens are packed as batch * seq_len rows, heads as
column blocks of head_dim.
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["rotary_frequencies", "rotate", "head_norm", "head_norm_backward", "diff_lambda", "diff_attention"]


def rotary_frequencies(rot_dim, base=10000.0, scaling="none", factor=1.0, original_len=4096, low_turns=1.0,
                       high_turns=None):
    """Radians per position of each pair, and the amplitude."""
    if high_turns is None:
        high_turns = 32.0 if scaling == "yarn" else 4.0
    i = np.arange(rot_dim // 2, dtype=np.float64)
    if scaling == "base" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = base ** (-2.0 * i / rot_dim)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "wavelength":
        turns = original_len * f / (2 * np.pi)
        keep = np.clip((turns - low_turns) / (high_turns - low_turns), 0, 1)
        return f * keep + f / factor * (1 - keep), 1.0
    if scaling == "yarn":
        def index(t):
            return rot_dim * math.log(original_len / (t * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(index(high_turns)), 0), min(math.ceil(index(low_turns)), rot_dim - 1)
        stretch = np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
        return f / factor * stretch + f * (1 - stretch), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def rotate(x, pos, freq, amp, hd, interleaved, inverse=False, absolute=False):
    """x [T, H * hd] turned; absolute: the sum of the magnitudes of each
    output's two terms, with cosine and sine taken as 1 (for error bounds)."""
    T, rot = x.shape[0], 2 * len(freq)
    y = np.array(x, np.float64).reshape(T, -1, hd)
    ang = np.asarray(pos, np.float64)[:, None] * freq[None, :]
    c, s = amp * np.cos(ang)[:, None], amp * np.sin(ang)[:, None] * (-1 if inverse else 1)
    ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    ib = ia + (1 if interleaved else rot // 2)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    if absolute:
        y = np.abs(y)
        y[..., ia] = y[..., ib] = amp * (np.abs(a) + np.abs(b))
    else:
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y.reshape(x.shape)


def head_norm(x, w, hd, eps):
    T = x.shape[0]
    x = np.asarray(x, np.float64).reshape(T, -1, hd)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return (x * r * np.asarray(w, np.float64)).reshape(T, -1)


def head_norm_backward(x, w, g, hd, eps):
    """g: gradient of the normed rows.  Returns dx, dw and, for error bounds,
    the magnitudes of the terms of each."""
    T = x.shape[0]
    x = np.asarray(x, np.float64).reshape(T, -1, hd)
    g = np.asarray(g, np.float64).reshape(T, -1, hd)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    h = g * np.asarray(w, np.float64)
    dx = r * (h - x * r * r * (h * x).mean(-1, keepdims=True))
    mx = r * (np.abs(h) + np.abs(x) * r * r * np.abs(h * x).mean(-1, keepdims=True))
    t = g * x * r
    return dx.reshape(T, -1), t.sum((0, 1)), mx.reshape(T, -1), np.abs(t).sum((0, 1))


def diff_lambda(lv, lambda_init):
    lq1, lk1, lq2, lk2 = (np.asarray(x, np.float64) for x in lv)
    e1, e2 = math.exp(lq1 @ lk1), math.exp(lq2 @ lk2)
    return e1 - e2 + lambda_init, e1, e2


def _weights(q, k, scale, causal):
    s = scale * (q @ k.T)
    if causal:
        s = np.where(np.arange(s.shape[1])[None, :] > np.arange(s.shape[0])[:, None], -np.inf, s)
    s = np.exp(s - s.max(-1, keepdims=True))
    return s / s.sum(-1, keepdims=True)


def diff_attention(q, k, v, lv, lambda_init, batch, heads, scale, causal, lens=None, da=None, rnd=0.0, stored=None):
    """Forward, and the backward when da is given.  Returns a dict of values
    and, under "bound", of error bounds for a kernel that keeps sums and
    statistics in fp32 and rounds its matrix operands (softmax weights, score
    gradients, the stored outputs) by at most ``rnd`` relative (0: not at all).
    ``stored``: the stored outputs are off by at most so much of their row's
    largest value instead.  The results' own rounding is not in the bounds."""
    kept = ((lambda x: rnd * np.abs(x)) if stored is None else
            (lambda x: np.zeros_like(x) + stored * np.abs(x).max(-1, keepdims=True)))
    hq, hkv, hd = heads
    T = q.shape[0]
    L = T // batch
    lens = [L] * batch if lens is None else lens
    lam, e1, e2 = diff_lambda(lv, lambda_init)
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    u = 2.0 ** -24
    res = {n: np.zeros_like(x) for n, x in (("a", q), ("dq", q), ("dk", k), ("dv", k))}
    bnd = {n: np.zeros_like(x) for n, x in res.items()}
    dlam = blam = 0.0
    for b in range(batch):
        n, r = int(lens[b]), slice(b * L, b * L + int(lens[b]))
        if n == 0:
            continue
        c32 = u * (n + 2 * hd + 32)          # a sum's worst case, and a few single operations
        for h in range(hq // 2):
            g = h * hkv // hq
            cv, ca = slice(2 * g * hd, 2 * (g + 1) * hd), slice(2 * h * hd, 2 * (h + 1) * hd)
            V = v[r, cv]
            P, O, Q, K, rel = [], [], [], [], []
            for m in (0, 1):
                Q.append(q[r, (2 * h + m) * hd:(2 * h + m + 1) * hd])
                K.append(k[r, (2 * g + m) * hd:(2 * g + m + 1) * hd])
                P.append(_weights(Q[m], K[m], scale, causal))
                O.append(P[m] @ V)
                # a weight's relative error: twice (score and log-sum-exp) the score's error
                rel.append(2 * u * ((hd + 8) * scale * (np.abs(Q[m]) @ np.abs(K[m]).T).max() + n + 16))
            res["a"][r, ca] = O[0] - lam * O[1]
            eO = [(rnd + rel[m] + c32) * (P[m] @ np.abs(V)) for m in (0, 1)]
            bnd["a"][r, ca] = eO[0] + abs(lam) * eO[1] + 4 * u * (np.abs(O[0]) + abs(lam) * np.abs(O[1]))
            if da is None:
                continue
            G = np.asarray(da, np.float64)[r, ca]
            dP, edP = G @ V.T, c32 * (np.abs(G) @ np.abs(V).T)
            res["dv"][r, cv] += (P[0] - lam * P[1]).T @ G
            W = P[0] * (rnd + rel[0] + c32) + abs(lam) * P[1] * (rnd + rel[1] + c32)
            bnd["dv"][r, cv] += W.T @ np.abs(G) + 4 * u * np.abs(res["dv"][r, cv])
            for m, coef in ((0, 1.0), (1, -lam)):
                D = (G * O[m]).sum(-1, keepdims=True)
                # D from the stored output and stored P_2 V
                st = kept(O[0] - lam * O[1]) + bnd["a"][r, ca] if m == 0 else 0.0
                st = st + (1 if m else 2 * abs(lam)) * (kept(O[1]) + eO[1])
                eD = (np.abs(G) * (st + c32 * (np.abs(O[0]) + (1 + abs(lam)) * np.abs(O[1])))).sum(-1, keepdims=True)
                E = P[m] * (dP - D)
                eE = P[m] * ((rel[m] + rnd) * np.abs(dP - D) + edP + eD + c32 * (np.abs(dP) + np.abs(D)))
                f = scale * abs(coef)
                cq, ck = slice((2 * h + m) * hd, (2 * h + m + 1) * hd), slice((2 * g + m) * hd, (2 * g + m + 1) * hd)
                res["dq"][r, cq] = coef * scale * (E @ K[m])
                bnd["dq"][r, cq] = f * ((eE + c32 * np.abs(E)) @ np.abs(K[m]))
                res["dk"][r, ck] += coef * scale * (E.T @ Q[m])
                bnd["dk"][r, ck] += f * ((eE + c32 * np.abs(E)).T @ np.abs(Q[m]))
                if m == 1:
                    dlam -= (P[1] * dP).sum()
                    blam += (P[1] * ((rel[1] + c32) * np.abs(dP) + edP)).sum()
    lq1, lk1, lq2, lk2 = (np.asarray(x, np.float64) for x in lv)
    for name, f, w in (("dlq1", e1, lk1), ("dlk1", e1, lq1), ("dlq2", -e2, lk2), ("dlk2", -e2, lq2)):
        res[name] = dlam * f * w
        bnd[name] = abs(f) * np.abs(w) * (blam + u * (2 * hd + 16) * abs(dlam))
    res["bound"] = bnd
    return res
