"""fp64 oracle of the dispatch to the experts, the way back, and their gradients.

Test infrastructure.  Not imported by the library.
"""
from __future__ import annotations

import numpy as np


def positions(idx, n_experts):
    """(offsets [E + 1], pair_pos [T, k]): pairs in (expert, t, i) order."""
    T, k = idx.shape
    keyed = sorted((int(idx[t, i]), t, i) for t in range(T) for i in range(k) if 0 <= idx[t, i] < n_experts)
    pos = np.full((T, k), -1, np.int64)
    offsets = np.zeros(n_experts + 1, np.int64)
    for at, (e, t, i) in enumerate(keyed):
        pos[t, i] = at
        offsets[e + 1:] += 1
    return offsets, pos


def combine_rows(rows, pair_pos, w=None, base=None):
    """(y, sum of the magnitudes of its terms)."""
    T, k = pair_pos.shape
    y = np.zeros((T, rows.shape[1])) if base is None else np.array(base, np.float64)
    mag = np.abs(y)
    for t in range(T):
        for i in range(k):
            if 0 <= pair_pos[t, i] < rows.shape[0]:
                term = (1.0 if w is None else w[t, i]) * rows[pair_pos[t, i]]
                y[t] += term
                mag[t] += np.abs(term)
    return y, mag


def combine_backward(dy, rows, pair_pos, w=None):
    """(drows, NaN where no pair's; dw; sum of the magnitudes of dw's terms)."""
    T, k = pair_pos.shape
    drows = np.full(rows.shape, np.nan)
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for i in range(k):
            p = pair_pos[t, i]
            if 0 <= p < rows.shape[0]:
                drows[p] = (1.0 if w is None else w[t, i]) * dy[t]
                dw[t, i] = (dy[t] * rows[p]).sum()
                mag[t, i] = np.abs(dy[t] * rows[p]).sum()
    return drows, dw, mag
