"""fp64 oracle of the microscaled 4-bit floats and of the products over them.

Test infrastructure.  Not imported by the library.  The format is the Open
Compute Project's MXFP4: 32 values share a power-of-two scale byte (bias 127,
255 = NaN); a value is a sign, a 2-bit exponent and a 1-bit mantissa.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32


def code_values():
    """The 16 values of a code, from its fields: sign, exponent e, mantissa m:
    e = 0: m / 2, else 2^(e-1) (1 + m / 2)."""
    v = np.empty(16)
    for c in range(16):
        e, m = (c >> 1) & 3, c & 1
        mag = m * 0.5 if e == 0 else 2.0 ** (e - 1) * (1 + 0.5 * m)
        v[c] = -mag if c & 8 else mag
    return v


def quantize(x):
    """x [..., cols] holding fp32 or bf16 values -> (codes [..., cols/2],
    scales [..., cols/32]).  Each value goes to the closest of the eight
    magnitudes by distance, of two equally close ones to the even code."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(x.shape[:-1] + (-1, BLOCK))
    bad = ~np.isfinite(b).all(-1)
    a = np.where(bad[..., None], 0.0, b)
    top = np.abs(a).max(-1)
    # frexp: top = f 2^e with 0.5 <= f < 1, so floor(log2 top) = e - 1
    e = np.where(top > 0, np.maximum(np.frexp(top)[1] - 1 - 2, -127), -127)
    m = np.ldexp(np.abs(a), -e[..., None])
    mags = code_values()[:8]
    dist = np.abs(m[..., None] - mags)
    near = dist.min(-1, keepdims=True)
    tied = dist == near
    odd_penalty = np.where(np.arange(8) % 2 == 0, 0, 1)
    code = np.where(tied, odd_penalty, 2).argmin(-1)     # even one first, then the odd one
    code = np.where(m > 6, 7, code)
    code = code + 8 * np.signbit(a)
    code = np.where(bad[..., None], 0, code).astype(np.uint8).reshape(x.shape)
    s = np.where(bad, 255, e + 127).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), s


def values(codes, scales):
    """float64 values [..., cols] of codes and scales."""
    codes = np.asarray(codes, dtype=np.uint8)
    c = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1,))
    v = code_values()[c].reshape(codes.shape[:-1] + (-1, BLOCK))
    s = np.asarray(scales, dtype=np.int64)
    v = np.ldexp(v, (s - 127)[..., None])
    v = np.where((s == 255)[..., None], np.nan, v)
    return v.reshape(codes.shape[:-1] + (-1,))


def silu(z):
    with np.errstate(over="ignore"):
        return z / (1.0 + np.exp(-z))


def product(a, w, offsets=None, src=None):
    """a [rows, K], w [G, N, K] float64 values; rows r of group g times w[g].
    src: a's row of every output row (out of range: zeros).  Returns (y [R, N],
    sum of the magnitudes [R, N], covered [R])."""
    R = len(src) if src is not None else a.shape[0]
    N = w.shape[1]
    y, mag, covered = np.zeros((R, N)), np.zeros((R, N)), np.zeros(R, bool)
    bounds = [0, R] if offsets is None else list(offsets)
    for g in range(w.shape[0]):
        rows = np.arange(bounds[g], bounds[g + 1])
        covered[rows] = True
        from_a = rows if src is None else np.asarray(src)[rows]
        here = (from_a >= 0) & (from_a < a.shape[0])
        y[rows[here]] = a[from_a[here]] @ w[g].T
        mag[rows[here]] = np.abs(a[from_a[here]]) @ np.abs(w[g].T)
    return y, mag, covered


def ffn_decode(x, gate_up, down, slot, w, shared_slot=-1):
    """y[t] = x[t] + sum_i w FFN_slot(x[t]) + FFN_shared(x[t]) over float64
    values gate_up [n, 2F, d] (gate rows even), down [n, d, F]; slots outside
    [0, n) add nothing."""
    n = gate_up.shape[0]

    def ffn(m, v):
        h = gate_up[m] @ v
        return down[m] @ (silu(h[0::2]) * h[1::2])

    y = np.array(x, dtype=np.float64)
    for t in range(x.shape[0]):
        for i in range(slot.shape[1]):
            if 0 <= slot[t, i] < n:
                y[t] += w[t, i] * ffn(slot[t, i], x[t])
        if shared_slot >= 0:
            y[t] += ffn(shared_slot, x[t])
    return y


def group_pairs(idx, n_experts):
    """(offsets, pair_pos, row_pair) of the pairs in (expert, t, i) order."""
    T, k = idx.shape
    pairs = [(idx[t, i], t * k + i) for t in range(T) for i in range(k)
             if 0 <= idx[t, i] < n_experts]
    pairs.sort()
    pos = np.full(T * k, -1, np.int32)
    for r, (_, p) in enumerate(pairs):
        pos[p] = r
    counts = np.bincount([e for e, _ in pairs], minlength=n_experts) if pairs else np.zeros(n_experts, int)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return offsets, pos.reshape(T, k), np.array([p for _, p in pairs], np.int32)
