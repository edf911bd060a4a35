"""GPU tests of the dispatch to the experts, the way back and their gradients
against the fp64 oracle.

Bars, u = 2^-24 (half a step of fp32).  Rows of the dispatch are copies: equal.
A sum of n fp32 terms added one after the other by fused multiply-adds rounds n
times, each time by at most u of a partial sum that the sum of the magnitudes
bounds: |y - ref| <= (n + 1) u mag; one rounding to the output's type adds
half a step of it.  dw sums d products in some order: (d + 1) u mag bounds any.
"""
import numpy as np
import pytest
import torch

import oracle.dispatch as od
from parity import need_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_STEP = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
F32, BF16 = torch.float32, torch.bfloat16


def _bf():
    import bit_expert_ffn_top_amd as bf
    return bf


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _idx(rng, T, k, E, dropped=0.0):
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]) if T else np.zeros((0, k))
    idx = np.where(rng.random((T, k)) < dropped, rng.choice([-1, E, -7, 2 ** 31 - 1, -2 ** 31], (T, k)), idx)
    return idx.astype(np.int32)


def _dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(need_gpu())
    return t if dtype is None else t.to(dtype)


def _randn(seed, shape, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).to(need_gpu())


def _check_dispatch(idx, E, d, dtype, seed=0):
    bf = _bf()
    T, k = idx.shape
    x = _randn(seed, (T, d), dtype)
    rows = torch.full((T * k, d), 7.5, dtype=dtype, device=x.device)
    f = bf.dispatch(x, _dev(idx), E, rows=rows)
    offsets, pos = od.positions(idx, E)
    assert np.array_equal(f.offsets.cpu().numpy(), offsets)
    assert np.array_equal(f.pair_pos.cpu().numpy(), pos)
    want = torch.full((T * k, d), 7.5, dtype=dtype)
    xc = x.cpu()
    for t in range(T):
        for i in range(k):
            if pos[t, i] >= 0:
                want[pos[t, i]] = xc[t]
    assert torch.equal(f.rows.cpu(), want)       # rows past the groups are left as they were
    return f


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,k,E,d,dropped", [
    (1, 1, 1, 4, 0.0), (1, 10, 512, 2048, 0.0), (2, 3, 5, 12, 0.3), (64, 10, 512, 256, 0.0),
    (65, 7, 60, 1044, 0.2), (131, 64, 64, 32, 0.5), (257, 1, 1024, 20, 0.1), (300, 8, 1000, 516, 1.0),
    (1025, 6, 33, 64, 0.2), (3000, 10, 128, 36, 0.1)])
def test_dispatch(T, k, E, d, dropped, dtype):
    rng = np.random.default_rng(T * 31 + k * 7 + E)
    _check_dispatch(_idx(rng, T, k, E, dropped), E, d, dtype)


@pytest.mark.parametrize("T", [40, 5000])
def test_dispatch_equal_ids_of_a_token(T):
    """A token that names an expert twice has two rows there, in k-slot order."""
    rng = np.random.default_rng(T)
    idx = rng.integers(-1, 9, (T, 6)).astype(np.int32)
    _check_dispatch(idx, 9, 8, F32)


@pytest.mark.parametrize("T", [300, 6000])
def test_dispatch_all_to_one_expert(T):
    idx = np.full((T, 2), 3, np.int32)
    idx[:, 1] = -1
    _check_dispatch(idx, 16, 64, BF16)


def test_dispatch_no_tokens():
    bf = _bf()
    f = bf.dispatch(torch.empty((0, 64), device=need_gpu()), _dev(np.zeros((0, 3), np.int32)), 5)
    assert f.rows.shape == (0, 64) and f.pair_pos.shape == (0, 3)
    assert f.offsets.cpu().tolist() == [0] * 6


@pytest.mark.parametrize("T,k,E", [(1, 10, 512), (64, 10, 512), (4097, 7, 60), (20000, 3, 1024), (65536, 2, 5)])
def test_dispatch_groups_as_group_pairs(T, k, E):
    """The same order as the grouping alone gives, up to the most tokens."""
    bf = _bf()
    rng = np.random.default_rng(T + E)
    idx = np.argsort(rng.random((T, E)), 1)[:, :k] if E < 100 else (rng.integers(0, E, (T, 1)) + 17 * np.arange(k)) % E
    idx = _dev(idx.astype(np.int32))
    x = _randn(1, (T, 8), BF16)
    f = bf.dispatch(x, idx, E)
    offsets, pos, row_pair = bf.group_pairs(idx, E)
    assert torch.equal(f.offsets, offsets) and torch.equal(f.pair_pos, pos)
    assert torch.equal(f.rows, x[(row_pair // k).long()])


def _pos(rng, T, k, R, missing):
    """Distinct rows for the pairs, some of them missing or out of range."""
    pos = rng.permutation(max(R, T * k))[:T * k].reshape(T, k)
    pos = np.where(pos >= R, -1, pos)
    bad = rng.choice([-1, R, R + 5, 2 ** 31 - 1, -2 ** 31], (T, k))
    return np.where(rng.random((T, k)) < missing, bad, pos).astype(np.int32)


SHAPES = [(1, 1, 4, 1, 0.0), (1, 10, 2048, 10, 0.0), (4, 10, 2048, 40, 0.1), (3, 2, 12, 9, 0.5), (37, 6, 1044, 222, 0.2),
          (130, 13, 264, 2000, 0.3), (65, 64, 100, 4160, 0.5), (2, 3, 16384, 6, 0.0), (700, 10, 72, 7000, 1.0)]


@pytest.mark.parametrize("types", [(F32, F32, F32), (BF16, BF16, BF16), (BF16, F32, F32), (F32, BF16, BF16),
                                   (BF16, None, F32), (F32, None, BF16), (BF16, F32, BF16), (F32, BF16, F32)])
@pytest.mark.parametrize("T,k,d,R,missing", SHAPES)
def test_combine_rows(T, k, d, R, missing, types):
    bf = _bf()
    rt, bt, yt = types
    rng = np.random.default_rng(T + 3 * k + d)
    pos = _pos(rng, T, k, R, missing)
    rows = _randn(1, (R, d), rt)
    base = None if bt is None else _randn(2, (T, d), bt)
    w = _randn(3, (T, k), F32)
    for weights in (w, None):
        y = bf.combine_rows(rows, _dev(pos), weights, base=base, dtype=yt)
        assert y.dtype == yt
        ref, mag = od.combine_rows(_np(rows), pos, None if weights is None else _np(w),
                                   None if base is None else _np(base))
        err = (k + 2) * U * mag
        assert (np.abs(_np(y) - ref) <= err + HALF_STEP[yt] * (np.abs(ref) + err)).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_combine_rows_in_place(dtype):
    bf = _bf()
    rng = np.random.default_rng(5)
    pos = _dev(_pos(rng, 50, 4, 200, 0.1))
    rows, base, w = _randn(1, (200, 132), BF16), _randn(2, (50, 132), dtype), _randn(3, (50, 4), F32)
    want = bf.combine_rows(rows, pos, w, base=base, dtype=dtype)
    assert bf.combine_rows(rows, pos, w, base=base, y=base) is base
    assert torch.equal(base, want)


def test_combine_rows_agrees_with_combine():
    """Bit for bit the older call where both apply."""
    bf = _bf()
    rng = np.random.default_rng(6)
    pos = _dev(_pos(rng, 90, 10, 900, 0.2))
    rows, base, w = _randn(1, (900, 256), F32), _randn(2, (90, 256), F32), _randn(3, (90, 10), F32)
    pos = torch.where(pos >= 900, -1, pos).int()
    assert torch.equal(bf.combine_rows(rows, pos, w, base=base), bf.combine(base, rows, pos, w))


@pytest.mark.parametrize("special", [float("inf"), float("-inf"), float("nan")])
def test_combine_rows_special_values(special):
    """A row with an infinity or NaN reaches its token only, a missing one none."""
    bf = _bf()
    rows = torch.ones((4, 16), dtype=BF16)
    rows[2, 5] = special
    pos = torch.tensor([[0, 2], [1, -1], [3, 4]], dtype=torch.int32)      # 4: past the rows
    y = bf.combine_rows(rows.to(need_gpu()), pos.to(need_gpu())).float().cpu()
    want = torch.tensor([[2.0], [1.0], [1.0]]).repeat(1, 16)
    want[0, 5] = special
    assert torch.equal(torch.nan_to_num(y, 1e4, 2e4, -2e4), torch.nan_to_num(want, 1e4, 2e4, -2e4))


@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("T,k,d,R,missing", SHAPES)
def test_combine_backward(T, k, d, R, missing, types):
    bf = _bf()
    gt, rt = types
    rng = np.random.default_rng(T + 5 * k + d)
    pos = _pos(rng, T, k, R, missing)
    dy, rows, w = _randn(1, (T, d), gt), _randn(2, (R, d), rt), _randn(3, (T, k), F32)
    drows = torch.full((R, d), 3.25, dtype=rt, device=dy.device)
    got, dw = bf.combine_backward(dy, rows, _dev(pos), w, drows=drows)
    assert got is drows
    ref, ref_w, mag = od.combine_backward(_np(dy), _np(rows), pos, _np(w))
    untouched = np.isnan(ref)
    assert (_np(drows)[untouched] == 3.25).all()
    ref = np.where(untouched, 3.25, ref)
    assert (np.abs(_np(drows) - ref) <= (U + HALF_STEP[rt] * (1 + U)) * np.abs(ref)).all()
    assert (np.abs(_np(dw) - ref_w) <= (d + 2) * U * mag).all()
    assert (_np(dw)[(pos < 0) | (pos >= R)] == 0).all()
    # each alone, and without weights: the same bits
    only = torch.full_like(drows, 3.25)
    assert torch.equal(bf.combine_backward(dy, None, _dev(pos), w, drows=only, need_w=False)[0], drows)
    none, dw2 = bf.combine_backward(dy, rows, _dev(pos), need_rows=False)
    assert none is None and torch.equal(dw2, dw)
    ones = bf.combine_backward(dy, rows, _dev(pos), torch.ones_like(w), drows=torch.zeros_like(drows))[0]
    assert torch.equal(bf.combine_backward(dy, rows, _dev(pos), drows=torch.zeros_like(drows), need_w=False)[0], ones)


def test_gradients_are_the_formulas_differences():
    """Central differences of <dy, combine(w, rows)> in single values of rows, w
    and x (through dispatch), in fp32: the sum is linear in each, so a difference
    of step 1 is the derivative but for the roundings of the two sums."""
    bf = _bf()
    rng = np.random.default_rng(11)
    T, k, E, d = 40, 3, 7, 24
    idx = _dev(_idx(rng, T, k, E, 0.1))
    x, dy, w = _randn(1, (T, d), F32), _randn(2, (T, d), F32), _randn(3, (T, k), F32)
    f = bf.dispatch(x, idx, E, rows=torch.zeros((T * k, d), device=x.device))
    drows, dw = bf.combine_backward(dy, f.rows, f.pair_pos, w, drows=torch.zeros_like(f.rows))
    dx = bf.dispatch_backward(drows, f.pair_pos)

    def loss(x=x, w=w, rows=None):
        if rows is None:
            rows = bf.dispatch(x, idx, E, rows=torch.zeros_like(f.rows)).rows
        return (bf.combine_rows(rows, f.pair_pos, w).double() * dy.double()).sum().item()

    scale = float((dy.abs().double().sum() * (f.rows.abs().max() + 1) * w.abs().max() * k).item())
    tol = 4 * (k + 2) * U * scale

    def difference(t, at, name):
        up, down = t.clone(), t.clone()
        up[at] += 1
        down[at] -= 1
        return (loss(**{name: up}) - loss(**{name: down})) / 2

    for at in [(0, 0), (3, 5), (39, 23), (17, 11)]:
        assert abs(difference(x, at, "x") - dx[at].item()) <= tol
        assert abs(difference(f.rows, at, "rows") - drows[at].item()) <= tol
    for at in [(0, 0), (5, 2), (39, 1)]:
        assert abs(difference(w, at, "w") - dw[at].item()) <= tol


def test_far_rows():
    """Rows whose byte offsets pass 2^32: the last rows of 4.3 GB."""
    bf = _bf()
    dev = need_gpu()
    R, d = 131_500, 16384
    rows = torch.zeros((R, d), dtype=BF16, device=dev)
    rows[-3:] = _randn(1, (3, d), BF16)
    pos = torch.tensor([[R - 1, 0], [R - 2, R - 3]], dtype=torch.int32, device=dev)
    assert R * d * 2 > 2 ** 32
    y = bf.combine_rows(rows, pos, dtype=F32)
    assert torch.equal(y[0], rows[-1].float()) and torch.equal(y[1], rows[-2].float() + rows[-3].float())
    dy = _randn(2, (2, d), BF16)
    drows, dw = bf.combine_backward(dy, rows, pos)
    assert torch.equal(drows[-1], dy[0]) and torch.equal(drows[-2], dy[1]) and torch.equal(drows[0], dy[0])
    ref = (dy[0].double() * rows[-1].double()).sum().item()
    mag = (dy[0].double() * rows[-1].double()).abs().sum().item()
    assert abs(dw[0, 0].item() - ref) <= (d + 2) * U * mag


def test_repeated_calls_give_the_same_bits():
    bf = _bf()
    rng = np.random.default_rng(8)
    idx = _dev(_idx(rng, 5000, 8, 64))
    x, dy, w = _randn(1, (5000, 96), BF16), _randn(2, (5000, 96), BF16), _randn(3, (5000, 8), F32)
    first = None
    for _ in range(3):
        f = bf.dispatch(x, idx, 64)
        y = bf.combine_rows(f.rows, f.pair_pos, w)
        drows, dw = bf.combine_backward(dy, f.rows, f.pair_pos, w)
        out = (*f, y, drows, dw, bf.dispatch_backward(drows, f.pair_pos))
        if first is not None:
            assert all(torch.equal(a, b) for a, b in zip(out, first))
        first = out


def test_no_rows():
    """Experts without any row: combine gives base, its gradient zeros."""
    bf = _bf()
    dev = need_gpu()
    pos, base, w = _dev(np.full((5, 3), -1, np.int32)), _randn(1, (5, 64), BF16), _randn(2, (5, 3), F32)
    rows = torch.empty((0, 64), dtype=BF16, device=dev)
    assert torch.equal(bf.combine_rows(rows, pos, w, base=base), base)
    assert torch.equal(bf.dispatch_backward(rows, pos, dtype=F32), torch.zeros((5, 64), device=dev))
    drows, dw = bf.combine_backward(base, rows, pos, w)
    assert drows.shape == (0, 64) and torch.equal(dw, torch.zeros_like(w))
    assert bf.combine_backward(base, rows, pos, w, need_w=False)[0].shape == (0, 64)
    pos0 = torch.empty((0, 3), dtype=torch.int32, device=dev)
    assert bf.combine_rows(_randn(3, (4, 64), F32), pos0).shape == (0, 64)
    drows, dw = bf.combine_backward(base[:0], _randn(3, (4, 64), F32), pos0)
    assert drows.shape == (4, 64) and dw.shape == (0, 3)


def test_more_threads_than_a_launch_has():
    """2.2 million tokens of 16,384 columns, 4.5 billion lanes' parts: rows from
    all over y, both ends and the seam between two launches among them."""
    bf = _bf()
    dev = need_gpu()
    T, d = 2_200_000, 16384
    assert T * (d // 8) > 2 ** 32
    rows = _randn(1, (3, d), BF16)
    w = torch.full((T, 1), 2.0, device=dev)
    pos = (torch.arange(T, device=dev) % 4).int()[:, None].contiguous()     # 3: no row
    y = bf.combine_rows(rows, pos, w)
    want = torch.cat([rows * 2, torch.zeros_like(rows[:1])])
    seam = 2 ** 31 // (d // 8)
    at = torch.tensor([0, 1, 2, 3, seam - 1, seam, seam + 1, 2 * seam - 1, 2 * seam, 2 * seam + 1, T - 2, T - 1], device=dev)
    assert torch.equal(y[at], want[(at % 4)])
