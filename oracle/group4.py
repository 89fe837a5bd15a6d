"""4-bit weights with a scale for each group of input channels, and their product with
16-bit rows (test infrastructure only).

  s = RNE16(fl32(max|w| / 7)) over a group;  r = fl32(1 / s);  c = clamp(rne(fl32(w * r)), -7, 7)
  (a group with an infinity or NaN: zero codes, a NaN scale)
  y = sum_g s_g * sum_{k in g} c_k x_k

The reference product is the exact sum in float64.  The device adds the exact products c x in
float32 and scales a group's sum into the row's: at most G additions in a group, counted at a
whole step (2^-23) each since the rounding inside a matrix instruction is not specified, then
K / G scaled additions and up to 16 of the parts of K at half a step, two more for the second order:
|error| <= (2 G + K / G + 18) 2^-24 sum_k |s c x|, above the float32 underflow.
"""
from __future__ import annotations

import numpy as np

from .numerics import from_f32, to_f32
from .quantizer import pack_int4


def pack(w_store, dtype: str, group: int):
    """(codes int8 [N x K], packed uint8 [N x K/2], scales in the storage type [N x K/group])."""
    w = to_f32(w_store, dtype)
    n, k = w.shape
    g = w.reshape(n, k // group, group)
    bad = ~np.isfinite(g).all(axis=2)
    g = np.where(bad[:, :, None], np.float32(0), g)
    s32 = (np.max(np.abs(g), axis=2) / np.float32(7.0)).astype(np.float32)
    s_store = from_f32(np.where(bad, np.float32("nan"), s32), dtype)
    s = to_f32(s_store, dtype)
    with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
        r = (np.float32(1.0) / s).astype(np.float32)
        r = np.where((s > 0) & np.isfinite(r), r, np.float32(0)).astype(np.float32)
    c = np.clip(np.rint((g * r[:, :, None]).astype(np.float32)), -7, 7).astype(np.int8).reshape(n, k)
    return c, pack_int4(c), s_store


def unpack(packed):
    """Signed values -8..7 of packed codes."""
    p = np.asarray(packed, dtype=np.uint8).astype(np.int16)
    c = np.empty(p.shape[:-1] + (2 * p.shape[-1],), dtype=np.int16)
    c[..., 0::2] = p & 15
    c[..., 1::2] = p >> 4
    return np.where(c > 7, c - 16, c)


def exact(x_store, dtype: str, packed, s_store, group: int):
    """(y float64, bound float64): the exact product and the largest error of the device's sums."""
    x = to_f32(x_store, dtype).astype(np.float64)
    w = unpack(packed) * np.repeat(to_f32(s_store, dtype).astype(np.float64), group, axis=1)
    k = x.shape[1]
    return x @ w.T, (2 * group + k // group + 18) * 2.0 ** -24 * (np.abs(x) @ np.abs(w).T)
