"""fp64 oracle of the low-rank adapters of many requests.

Test infrastructure.  Not imported by the library.
"""
from __future__ import annotations

import numpy as np


def requests_of(T, seq_offsets):
    """Request of every row, -1 for none: bounds clamped to [0, T], one below an
    earlier one counts as that one; without bounds a row is a request."""
    if seq_offsets is None:
        return np.arange(T)
    bounds = np.maximum.accumulate(np.clip(np.asarray(seq_offsets, np.int64), 0, T))
    out = np.full(T, -1)
    for s in range(len(bounds) - 1):
        out[bounds[s]:bounds[s + 1]] = s
    return out


def lora(base, x, a, b, adapter, seq_offsets=None, scale=None):
    """dict of y (NaN in rows of no request), h [T, rank] (scaled), h_mag and
    y_mag (the same sums over magnitudes), b_of (|b| of the row's adapter, or None)."""
    T, n, rank = x.shape[0], a.shape[0], a.shape[1]
    y = np.array(base, np.float64)
    h, h_mag = np.zeros((T, rank)), np.zeros((T, rank))
    y_mag = np.abs(y)
    b_of = [None] * T
    for t, s in enumerate(requests_of(T, seq_offsets)):
        if s < 0:
            y[t] = np.nan
            continue
        m = int(adapter[s])
        if 0 <= m < n:
            f = 1.0 if scale is None else float(scale[m])
            h[t] = f * (a[m] @ x[t])
            h_mag[t] = abs(f) * (np.abs(a[m]) @ np.abs(x[t]))
            y[t] += b[m] @ h[t]
            y_mag[t] += np.abs(b[m]) @ np.abs(h[t])
            b_of[t] = np.abs(b[m])
    return dict(y=y, h=h, h_mag=h_mag, y_mag=y_mag, b_of=b_of)
