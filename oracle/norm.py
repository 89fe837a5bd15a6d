"""Root-mean-square norm with the residual's addition, and its quantized form (test
infrastructure only).

  h = RNE16(fl32(x + r));  q = sum_k h^2 / K;  rstd = fl32(1 / sqrt(q + eps))
  v = fl32(fl32(h * rstd) * w);  y = RNE16(v), or the row quantizer's codes of v

The sum, the division and the root are float64: squares of 16-bit values are exact there,
so the float32 rstd is that of the exact sum short of a tie at 2^-53.
"""
from __future__ import annotations

import numpy as np

from .numerics import from_f32, to_f32
from .quantizer import qmax, quantize_groups, quantize_static, split_dual


def rows(x_store, dtype: str, weight=None, eps: float = 1e-6, res_store=None):
    """(h in the storage type, v float32); weight: float32 [K] or None for ones."""
    x = to_f32(x_store, dtype)
    with np.errstate(all="ignore"):
        h_store = np.asarray(x_store) if res_store is None else from_f32(x + to_f32(res_store, dtype), dtype)
        h = to_f32(h_store, dtype)
        q = np.sum(h.astype(np.float64) ** 2, axis=1, keepdims=True) / h.shape[1]
        rstd = (1.0 / np.sqrt(q + eps)).astype(np.float32)
        v = (h * rstd).astype(np.float32)
        if weight is not None:
            v = (v * np.asarray(weight, dtype=np.float32)[None, :]).astype(np.float32)
    return h_store, v


def quant(v: np.ndarray, bits: int, out_idx=None, static_scale=None):
    """Codes and scales of the normed rows, per token or static, with the outlier partition."""
    Q = qmax(bits)
    parts = [v] if out_idx is None or len(out_idx) == 0 else list(split_dual(v, out_idx))
    codes, scales = [], []
    for i, p in enumerate(parts):
        if static_scale is None:
            c, s = quantize_groups(p, Q, axis=1)
        else:
            c, s = quantize_static(p, Q, np.asarray(static_scale, dtype=np.float32).reshape(-1)[i])
            s = np.array([s], dtype=np.float32)
        codes.append(c)
        scales.append(np.asarray(s, dtype=np.float32))
    codes = np.concatenate(codes, axis=1)
    if len(parts) == 1:
        return codes, scales[0]
    return codes, np.stack(scales, axis=1) if static_scale is None else np.concatenate(scales)
