"""Routing to experts and the way back (test infrastructure only).

Row by row, choice by choice, in float64: scores p (softmax or sigmoid), c = p + bias (the scores
themselves without a bias) for the choice, groups by the sum of their best one or two, ties to the
lower index, weights p / sum p.  Closed experts (score or bias -inf) are never chosen (a bias leaves p
as it is); a row with a NaN (or, for softmax, an infinite score) is not routed and has NaN weights.
"""
from __future__ import annotations

import numpy as np

F = np.float32


def choose(x, top, score="softmax", bias=None, groups=1, keep=None, best=1, renorm=True, scale=1.0):
    """One row of float64 scores: (experts list, weights float64 list), -1 and 0 where none is open."""
    x = np.asarray(x, np.float64)
    e = len(x)
    keep = groups if keep is None else keep
    with np.errstate(all="ignore"):
        if score == "softmax":
            m = np.max(x)
            p = np.exp(x - m) if m > -np.inf else np.zeros(e)
            p = p / p.sum() if p.sum() > 0 else p
        else:
            p = 1.0 / (1.0 + np.exp(-x))
        c = x.copy() if bias is None else np.where(x == -np.inf, -np.inf, p + np.asarray(bias, np.float64))
    if np.isnan(x).any() or np.isnan(c).any() or (score == "softmax" and (x == np.inf).any()):
        return [-1] * top, [np.nan] * top
    open_ = c > -np.inf
    if groups > 1:
        size = e // groups
        by = np.where(open_, p, -np.inf) if best == 2 and bias is None else c
        marks = []
        for g in range(groups):
            s = sorted(by[g * size:(g + 1) * size], reverse=True)
            marks.append(s[0] + (s[1] if best == 2 and s[1] > -np.inf else 0.0))
        kept = sorted(range(groups), key=lambda g: (-marks[g], g))[:keep]
        open_ &= np.isin(np.arange(e) // size, kept)
    order = sorted((i for i in range(e) if open_[i]), key=lambda i: (-c[i], i))[:top]
    w = [p[i] for i in order]
    total = sum(w)
    if renorm:
        w = [v / total if total > 0 else 0.0 for v in w]
    none = top - len(order)
    return order + [-1] * none, [v * scale for v in w] + [0.0] * none


def route(x, top, **how):
    """(offsets, rows, weights float64, experts, place) of float64 scores [m x e]."""
    m, e = x.shape
    got = [choose(r, top, **how) for r in x]
    chosen = np.array([g[0] for g in got], np.int32).reshape(m, top)
    weights = np.array([g[1] for g in got], np.float64).reshape(m, top)
    place = np.full((m, top), -1, np.int32)
    rows = np.full(m * top, -1, np.int32)
    offsets, n = [0], 0
    for i in range(e):
        for t, j in zip(*np.nonzero(chosen == i)):
            place[t, j], rows[n] = n, t
            n += 1
        offsets.append(n)
    return np.array(offsets, np.int32), rows, weights, chosen, place


def combine(y, place, weights, res=None, gate=None, at=None):
    """float32 outputs, one rounding a step, before the output's: y, res, gate float32; at: each row's set."""
    m, top = place.shape
    v = np.zeros((m, y.shape[1]), F)
    with np.errstate(all="ignore"):
        for j in range(top):
            p = place[:, j]
            ok = (p >= 0) & (p < len(y))
            q = np.where(ok[:, None], y[np.where(ok, p, 0)] if len(y) else F(0), F(0)).astype(F)
            v = (v + (q * weights[:, j].astype(F)[:, None]).astype(F)).astype(F)
        if gate is None:
            return v if res is None else (v + res).astype(F)
        ok = (at >= 0) & (at < len(gate))
        v = (v * gate[np.where(ok, at, 0)].astype(F)).astype(F)
        v = v if res is None else (v + res).astype(F)
        return np.where(ok[:, None], v, F(0) if res is None else res).astype(F)
