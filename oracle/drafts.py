"""fp64 oracle of the verification of drafted tokens.

Test infrastructure.  Not imported by the library.
"""
from __future__ import annotations

import math

import numpy as np


def _draw(r, u):
    """The smallest v whose sum r[0] + .. + r[v] lies above u times the whole sum,
    the last v with r[v] > 0 if there is none, -1 if r is nothing but zeros; u below
    0 counts as 0."""
    some = np.nonzero(r > 0)[0]
    if len(some) == 0:
        return -1
    want = (0.0 if u < 0 else u) * math.fsum(r)
    cum = np.cumsum(r)
    over = np.nonzero(cum > want)[0]
    return int(over[0]) if len(over) else int(some[-1])


def _counted(r):
    with np.errstate(invalid="ignore"):
        return np.where((r > 0) & np.isfinite(r), r, 0.0)


def verify(p, q, draft, u_accept, u_sample, n_draft=None):
    """(tokens [B, n + 1], n_accepted [B])."""
    B, n = draft.shape
    V = p.shape[2]
    tokens = np.full((B, n + 1), -1, np.int64)
    accepted = np.zeros(B, np.int64)
    for s in range(B):
        m = n if n_draft is None else min(max(int(n_draft[s]), 0), n)
        j = 0
        while j < m:
            x = int(draft[s, j])
            if not 0 <= x < V:
                break
            qx = 1.0 if q is None else float(q[s, j, x])
            if not float(u_accept[s, j]) * qx < float(p[s, j, x]):
                break
            tokens[s, j] = x
            j += 1
        accepted[s] = j
        whole = np.asarray(p[s, j], np.float64)
        with np.errstate(invalid="ignore"):
            if j == m:
                r = _counted(whole)
            elif q is not None:
                r = _counted(whole - np.asarray(q[s, j], np.float64))
            else:
                r = _counted(whole)
                if 0 <= draft[s, j] < V:
                    r[draft[s, j]] = 0.0
        if not (r > 0).any():
            r = _counted(whole)
        tokens[s, j] = _draw(r, float(u_sample[s]))
    return tokens, accepted
