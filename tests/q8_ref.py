"""Plain 64-bit forms of the 8-bit products with token and channel scales and
of the scored router, for the tests that compare the kernels with them."""
from __future__ import annotations

import numpy as np


def quant(x: np.ndarray):
    """Codes and scales of x [T, n] (values of its type, exact in float64; their
    largest is a float32)."""
    x = x.astype(np.float64)
    a = np.abs(x).max(axis=1)
    with np.errstate(all="ignore"):
        bad = ~np.isfinite(x).all(axis=1)
        s = a.astype(np.float32) * (np.float32(1) / np.float32(127))  # one product in binary32
        s64 = s.astype(np.float64)[:, None]
        r = np.where(s64 > 0, x / np.where(s64 > 0, s64, 1.0), 0.0).astype(np.float32)
        q = np.clip(np.rint(r.astype(np.float64)), -127, 127)
    q[bad] = 0
    s[bad] = np.nan
    return q.astype(np.int8), s


def swiglu(g: np.ndarray, u: np.ndarray) -> np.ndarray:
    g, u = g.astype(np.float64), u.astype(np.float64)
    with np.errstate(all="ignore"):
        return (g / (1.0 + np.exp(-g)) * u).astype(np.float32)


def product(q, s, w, ws, bias=None) -> np.ndarray:
    """[T, N] in float64; the integer sums are exact (below 2^53)."""
    acc = q.astype(np.float64) @ w.astype(np.float64).T
    y = acc * s.astype(np.float64)[:, None] * ws.astype(np.float64)[None, :]
    return y if bias is None else y + bias.astype(np.float64)[None, :]


def tables(idx: np.ndarray, E: int):
    """coli_moe_dispatch's offs [E + 1] and perm [T * k] of idx [T, k]."""
    flat = idx.ravel()
    perm = np.concatenate([np.flatnonzero(flat == e) for e in range(E)] + [np.flatnonzero(flat < 0)])
    counts = np.array([(flat == e).sum() for e in range(E)])
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), perm.astype(np.int32)


def route(logits, bias, k, G=1, TG=1, score="sigmoid", group_score="top2", norm=True, rsf=1.0):
    """idx [T, k] and w [T, k] (float64) by the definition, expert by expert."""
    T, E = logits.shape
    per = E // G
    idx = np.full((T, k), -1, dtype=np.int64)
    w = np.zeros((T, k))
    for t in range(T):
        l = logits[t].astype(np.float64)
        off = np.isnan(l) | (l == -np.inf)
        p = np.zeros(E)
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                p[~off] = 1.0 / (1.0 + np.exp(-l[~off]))
        elif (~off).any():
            top = l[~off].max()
            with np.errstate(invalid="ignore"):
                e = np.where(l[~off] == top, 1.0, np.exp(l[~off] - top))
            p[~off] = e / e.sum()
        p32 = p.astype(np.float32)
        c = p32 if bias is None else p32 + bias
        c = np.where(off | np.isnan(c), -np.inf, c).astype(np.float32)
        if TG < G:
            gs = np.full(G, -np.inf, dtype=np.float32)
            for g in range(G):
                v = np.sort(c[g * per:(g + 1) * per])[::-1]
                gs[g] = v[0]
                if group_score == "top2" and per > 1 and v[1] > -np.inf:
                    gs[g] = np.float32(v[0] + v[1])
            kept = sorted(range(G), key=lambda g: (-gs[g], g))[:TG]
            for g in range(G):
                if g not in kept:
                    c[g * per:(g + 1) * per] = -np.inf
        order = sorted(range(E), key=lambda e: (-c[e], e))[:k]
        order = [e for e in order if c[e] > -np.inf]
        idx[t, :len(order)] = order
        v = p32[order].astype(np.float64)
        if norm:
            v = v / v.sum() if len(order) and v.sum() > 0 else np.zeros(len(order))
        w[t, :len(order)] = v * rsf
    return idx, w
