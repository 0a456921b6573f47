"""Plain fp64 definitions of rows in 8 bits and of what is formed from them.

TEST INFRASTRUCTURE ONLY, as ``kfac_oracle``: NumPy, from the formulas of include/kfac.h,
sharing no code with the HIP library. Inputs are the exact values of the arrays that the
library was given. Pinned in ``tests/test_q8_oracle.py`` by brute force and closed forms.
"""
import math

import numpy as np

__all__ = ["quantize_rows", "row_values", "linear", "weight_grad", "factor_packed"]


def _scale(m, pow2):
    if not math.isfinite(m):
        return math.nan
    if m == 0.0:
        return 1.0
    if not pow2:
        return max(float(np.float32(np.float32(m) / np.float32(127))), 2.0 ** -126)
    e = -126
    while 127 * 2.0 ** e < m:
        e += 1
    return 2.0 ** e


def quantize_rows(x, mask=None, pow2=True):
    """(q as fp64 whole numbers, scale in fp64) of every row."""
    x = np.asarray(x, dtype=np.float64)
    q, scale = np.zeros(x.shape), np.zeros(x.shape[0])
    for t, row in enumerate(x):
        if mask is not None and not mask[t]:
            continue
        m = float(np.abs(row).max()) if row.size else 0.0
        s = scale[t] = _scale(m if not np.isnan(row).any() else math.nan, pow2)
        if math.isnan(s):
            continue
        v = row / s
        low = np.floor(v)
        up = (v - low > 0.5) | ((v - low == 0.5) & (low % 2 == 1))
        most = 63 if pow2 and s >= 2.0 ** 122 else 127
        q[t] = np.clip(low + up, -most, most)
    return q, scale


def row_values(q, scale):
    """scale[t] q[t], zeros where scale is 0."""
    return np.asarray(q, dtype=np.float64) * np.asarray(scale, dtype=np.float64)[:, None]


def linear(q, scale, w, w_scale, bias=None):
    """y, and the sum of the magnitudes that it is made of."""
    acc = np.asarray(q, dtype=np.float64) @ np.asarray(w, dtype=np.float64).T
    part = acc * np.asarray(scale, dtype=np.float64)[:, None] * np.asarray(w_scale, dtype=np.float64)
    b = np.zeros(part.shape[1]) if bias is None else np.asarray(bias, dtype=np.float64)
    return part + b, np.abs(part) + np.abs(b)


def weight_grad(g, q, scale):
    """dW, db and the sums of the magnitudes of their terms."""
    live = np.asarray(scale) != 0
    g, a = np.asarray(g, dtype=np.float64)[live], row_values(q, scale)[live]
    return g.T @ a, g.sum(0), np.abs(g).T @ np.abs(a), np.abs(g).sum(0)


def factor_packed(q, scale, bias, old=None, decay=0.0):
    """The packed factor (upper triangle row by row), and the same of the magnitudes of its terms."""
    live = np.asarray(scale) != 0
    a = row_values(q, scale)[live]
    if bias:
        a = np.concatenate([a, np.ones((a.shape[0], 1))], 1)
    i, j = np.triu_indices(a.shape[1])
    if not len(a):
        kept = np.zeros(len(i)) if decay == 0.0 else np.asarray(old, dtype=np.float64)
        return kept, np.abs(kept)
    new, size = (a.T @ a)[i, j] / len(a), (np.abs(a).T @ np.abs(a))[i, j] / len(a)
    if decay != 0.0:
        old = np.asarray(old, dtype=np.float64)
        new, size = decay * old + (1 - decay) * new, decay * np.abs(old) + (1 - decay) * size
    return new, size
