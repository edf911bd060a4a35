"""fp64 oracle of the router's balance and z losses, per-expert counts, and of
the gradient of the logits.

Test infrastructure.  Not imported by the library.
"""
from __future__ import annotations

import numpy as np


def softmax(row):
    """(p, lse) of one row: NaN as -inf, the difference of two equal values
    (infinities too) as 0."""
    v = np.where(np.isnan(row), -np.inf, np.asarray(row, dtype=np.float64))
    m = v.max()
    with np.errstate(invalid="ignore"):
        d = np.where(v == m, 0.0, v - m)
    e = np.exp(d)
    return e / e.sum(), m + np.log(e.sum())


def rows_of(T, seq_offsets, n_seq, mask):
    """The rows of every sequence that take part."""
    off = [0, T] if seq_offsets is None else [min(max(int(o), 0), T) for o in seq_offsets]
    return [[t for t in range(off[s], off[s + 1]) if mask is None or mask[t]] for s in range(n_seq)]


def route_balance(logits, idx, seq_offsets=None, mask=None):
    """dict of balance, z [S], counts, prob_sum [S, E], n_tokens [S]."""
    T, E = logits.shape
    k = idx.shape[1]
    S = 1 if seq_offsets is None else len(seq_offsets) - 1
    counts, psum = np.zeros((S, E), np.int64), np.zeros((S, E))
    balance, z, n = np.zeros(S), np.zeros(S), np.zeros(S, np.int64)
    for s, rows in enumerate(rows_of(T, seq_offsets, S, mask)):
        n[s] = len(rows)
        for t in rows:
            p, lse = softmax(logits[t])
            psum[s] += p
            if np.isfinite(lse):
                z[s] += lse * lse
            for e in idx[t]:
                if 0 <= e < E:
                    counts[s, e] += 1
        if rows:
            balance[s] = E / (k * len(rows) ** 2) * (counts[s] * psum[s]).sum()
            z[s] /= len(rows)
    return dict(balance=balance, z=z, counts=counts, prob_sum=psum, n_tokens=n)


def route_backward(logits, idx, counts=None, n_tokens=None, g_balance=None, g_z=None, w=None,
                   dw=None, seq_offsets=None, mask=None):
    """dlogits [T, E] by the three terms of the formula."""
    T, E = logits.shape
    k = idx.shape[1]
    S = 1 if seq_offsets is None else len(seq_offsets) - 1
    out = np.zeros((T, E))
    for s, rows in enumerate(rows_of(T, seq_offsets, S, mask)):
        n = int(n_tokens[s]) if n_tokens is not None else 0
        for t in rows:
            if n > 0 and (g_balance is not None or g_z is not None):
                p, lse = softmax(logits[t])
                if g_balance is not None:
                    c = counts[s].astype(np.float64)
                    out[t] += g_balance[s] * E / (k * n * n) * p * (c - (c * p).sum())
                if g_z is not None and np.isfinite(lse):
                    out[t] += g_z[s] * 2.0 / n * lse * p
            if w is not None:
                dot = (w[t] * dw[t]).sum()
                for i in range(k):
                    if 0 <= idx[t, i] < E:
                        out[t, idx[t, i]] += w[t, i] * (dw[t, i] - dot)
    return out
