"""Products of several experts: rows sorted by expert, each against its own expert's
weights (test infrastructure only).  The integer form's rows equal the single layer's
(gemm.py), the 16-bit form's the unquantized layer's (dense.py)."""
from __future__ import annotations

import numpy as np


def apply(offsets, rows, t, n, one):
    """float64 [t x n] with NaN where no expert owns the row.

    one(e, idx): expert e's float64 outputs for the rows idx of the operand (all valid);
    an index of `rows` outside the operand, -1 here, gives zeros."""
    y = np.full((t, n), np.nan)
    for e in range(len(offsets) - 1):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi <= lo:
            continue
        idx = np.arange(lo, hi) if rows is None else np.asarray(rows)[lo:hi]
        out = np.zeros((hi - lo, n))
        ok = idx >= 0
        if ok.any():
            out[ok] = one(e, idx[ok])
        y[lo:hi] = out
    return y
