"""Low-rank adapters beside a shared projection (test infrastructure only).

  delta[i] = scale[a] * (x[i] . down[a]^T) . up[a]^T in float64, a = index[i], 0 without an adapter

and the bound on a kernel that sums in float32 and passes t = scale * x . down^T on in two 16-bit
pieces: an addition is counted at 2^-23 (K of them for t, two R for the output), t's own
rounding and that of the pieces (bf16 2^-16 of t, nothing for a float32 output, which takes three pieces;
fp16 2^-22 of t, and 2^-38 of the row's largest where a piece is below fp16's normal range).
"""
from __future__ import annotations

import numpy as np


def exact(x, down, up, index, scale=None, dtype="bf16", out=None):
    """float64 (delta, bound) [m x n]; x, down, up float64 arrays; out: the output's type, dtype or "fp32"."""
    m, n = len(x), up.shape[1]
    k, r = x.shape[1], down.shape[1]
    delta, bound = np.zeros((m, n)), np.zeros((m, n))
    with np.errstate(all="ignore"):
        for a in range(len(down)):
            at = np.nonzero(np.asarray(index) == a)[0]
            if not len(at):
                continue
            s = 1.0 if scale is None else float(scale[a])
            t = s * (x[at] @ down[a].T)
            ta = abs(s) * (np.abs(x[at]) @ np.abs(down[a]).T)
            ua = np.abs(up[a]).T
            delta[at] = t @ up[a].T
            sums = np.abs(t) @ ua
            bound[at] = (2 * k + 10) * 2.0 ** -24 * (ta @ ua) + (4 * r + 4) * 2.0 ** -24 * sums
            if dtype == "bf16":
                bound[at] += 0.0 if out == "fp32" else 2.0 ** -16 * sums
            else:
                bound[at] += 2.0 ** -22 * sums + 2.0 ** -38 * np.abs(t).max(1, keepdims=True) * ua.sum(0)[None, :]
    return delta, bound
