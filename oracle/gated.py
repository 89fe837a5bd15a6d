"""Norms before and after a block with its gate and residual scale (test infrastructure only).

  u = y, or the post norm of y;  s = RNE16(fl32(h + fl32(u * fl32(g * alpha))))
  v = norm(s) * w;  v = fl32(fl32(v * fl32(1 + c)) + d)

A norm is fl32(fl32(x - mean) * rstd), mean = fl32(sum x / K) for "layer" and 0 for "rms", rstd =
fl32(1 / sqrt(sum (x - sum x / K)^2 / K + eps)), the moments in float64 (two passes here).
``sets`` gives each row's set of gate, scale and shift; one outside them is a row without any.
"""
from __future__ import annotations

import numpy as np

from .numerics import from_f32, to_f32

F = np.float32


def normed(x: np.ndarray, kind: str, eps: float, weight=None) -> np.ndarray:
    """float32 rows -> float32 rows."""
    d = x.astype(np.float64)
    k = x.shape[1]
    mu = np.sum(d, axis=1, keepdims=True) / k if kind == "layer" else np.zeros((len(x), 1))
    q = np.sum((d - mu) ** 2, axis=1, keepdims=True) / k
    v = ((x - mu.astype(F)).astype(F) * (1.0 / np.sqrt(q + eps)).astype(F)).astype(F)
    return v if weight is None else (v * np.asarray(weight, F)[None, :]).astype(F)


def row_sets(m: int, sets: int, index=None) -> np.ndarray:
    """Each row's set: index, or an even split."""
    return np.arange(m) // (m // sets) if index is None else np.asarray(index).astype(np.int64)


def rows(y_store, h_store, dtype: str, norm: str = "rms", weight=None, eps: float = 1e-6, post=None, post_weight=None,
         alpha: float = 1.0, gate=None, scale=None, shift=None, index=None):
    """(s in the storage type, v float32); gate, scale, shift: float32 [sets x K] or None."""
    m = np.shape(h_store)[0]
    mods = [t for t in (gate, scale, shift) if t is not None]
    sets = mods[0].shape[0] if mods else 1
    at = row_sets(m, sets, index)
    ok = ((at >= 0) & (at < sets))[:, None]
    at = np.where(ok[:, 0], at, 0)
    s_store = np.asarray(h_store)
    with np.errstate(all="ignore"):
        if y_store is not None:
            h, u = to_f32(h_store, dtype), to_f32(y_store, dtype)
            if post is not None:
                u = normed(u, post, eps, post_weight)
            g = np.full((m, 1), F(alpha)) if gate is None else (gate[at].astype(F) * F(alpha)).astype(F)
            s = (h + (u * g).astype(F)).astype(F)
            s_store = np.where(ok, from_f32(s, dtype), s_store)
        v = normed(to_f32(s_store, dtype), norm, eps, weight)
        if scale is not None:
            v = np.where(ok, (v * (F(1) + scale[at].astype(F)).astype(F)).astype(F), v)
        if shift is not None:
            v = np.where(ok, (v + shift[at].astype(F)).astype(F), v)
    return s_store, v
