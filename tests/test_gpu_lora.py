"""GPU tests of the low-rank adapters of many requests against the fp64 oracle.

Bars, u = 2^-24.  h = A x sums d_in products in fp32: each addition is off by at
most a step 2u of a partial sum that the sum of the magnitudes bounds, so
|dh| <= 2 (d_in + 8) u h_mag, the scale's rounding and the parts of an fp32 x
that a product may round among the 8.  h itself may be kept as a sum of bfloat16
parts, three for fp32 results (off by 2^-24 of it) and two for bfloat16 ones
(2^-16).  B h sums rank products and base the same way.  One rounding to the
output's type adds half a step of it.
"""
import numpy as np
import pytest
import torch

import oracle.lora as ol
from parity import need_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
HALF_STEP = {F32: U, BF16: 2.0 ** -8}
H_PARTS = {F32: 2.0 ** -24, BF16: 2.0 ** -16}


def _bf():
    import bit_expert_ffn_top_amd as bf
    return bf


def _np(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def _i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=need_gpu())


def _inputs(T, n, rank, d_in, d_out, xt, yt, seed=0):
    dev = need_gpu()
    g = torch.Generator().manual_seed(seed + T * 7 + rank)

    def randn(*shape):
        return torch.randn(shape, generator=g)

    x = (randn(T, d_in) * torch.exp(randn(T, 1))).to(xt).to(dev)
    base = randn(T, d_out).to(yt).to(dev)
    a = (randn(n, rank, d_in) / d_in ** 0.5).to(BF16).to(dev)
    b = (randn(n, d_out, rank) / rank ** 0.5).to(BF16).to(dev)
    return base, x, a, b, (0.5 + torch.rand((n,), generator=g)).to(dev)


def _bound(r, d_in, rank, yt):
    dh = 2 * (d_in + 8) * U * r["h_mag"] + H_PARTS[yt] * np.abs(r["h"])
    err = 2 * (rank + 8) * U * r["y_mag"]
    for t, bm in enumerate(r["b_of"]):
        if bm is not None:
            err[t] += 1.001 * (bm @ dh[t])
    return err + HALF_STEP[yt] * (np.abs(r["y"]) + err)


def _check(base, x, a, b, adapter, seq, scale):
    bf = _bf()
    y = torch.full_like(base, 9.5)
    bf.lora(base, x, a, b, _i32(adapter), seq_offsets=None if seq is None else _i32(seq), scale=scale, y=y)
    r = ol.lora(_np(base), _np(x), _np(a), _np(b), adapter, seq, _np(scale))
    none = np.isnan(r["y"])
    assert (_np(y)[none] == 9.5).all()            # rows of no request: left as they were
    plain = np.array([bm is None for bm in r["b_of"]])[:, None] & ~none
    assert (_np(y)[plain] == _np(base)[plain]).all()
    ok = np.abs(_np(y) - r["y"]) <= _bound(r, x.shape[1], a.shape[1], base.dtype)
    assert (ok | none).all(), np.argwhere(~(ok | none))[:5]
    # in place: the same bits
    mine = base.clone()
    out = bf.lora(mine, x, a, b, _i32(adapter), seq_offsets=None if seq is None else _i32(seq), scale=scale, y=mine)
    assert out is mine
    assert torch.equal(mine[torch.from_numpy(~none[:, 0]).to(mine.device)],
                       y[torch.from_numpy(~none[:, 0]).to(mine.device)])
    return y


TYPES = [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("T,n,rank,d_in,d_out", [
    (1, 1, 8, 32, 16), (1, 16, 16, 2048, 1536), (2, 3, 24, 96, 48), (17, 5, 32, 224, 80), (64, 48, 16, 2048, 1536),
    (70, 1, 64, 512, 1040), (33, 9, 128, 1056, 272), (5, 2, 40, 16384, 32), (3, 2, 16, 64, 16384),
    (300, 7, 8, 160, 64)])
def test_a_row_for_every_request(T, n, rank, d_in, d_out, types):
    base, x, a, b, scale = _inputs(T, n, rank, d_in, d_out, *types)
    adapter = np.random.default_rng(T).integers(-1, n + 1, T)      # -1 and n: without one
    _check(base, x, a, b, adapter, None, scale)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("bounds,T", [
    ([0, 1], 1), ([0, 5, 5, 21, 40], 40), ([0, 16, 32, 64], 64), ([3, 20, 50], 60), ([0, 0, 0, 7, 7], 7),
    ([0, 300, 301, 302, 700], 700), ([0, 15, 31, 48, 49, 66, 129, 193, 258], 258), ([0, 1000], 1000)])
@pytest.mark.parametrize("rank,d_in,d_out", [(16, 256, 144), (72, 96, 400)])
def test_ragged_requests(bounds, T, rank, d_in, d_out, types):
    n = 4
    base, x, a, b, scale = _inputs(T, n, rank, d_in, d_out, *types)
    adapter = np.random.default_rng(T + len(bounds)).integers(-1, n, len(bounds) - 1)
    _check(base, x, a, b, adapter, bounds, scale)


@pytest.mark.parametrize("bounds", [[0, 30, 20, 40], [-5, 10, 99], [50, 10, 5], [7, 3, 9, 4, 30, 2 ** 31 - 1],
                                    [0, 0], [40, 40], [-2 ** 31, 12, -9, 33]])
def test_bounds_out_of_order_or_range(bounds):
    """A bound below an earlier one counts as that one, bounds past the rows as
    the last row's end: no row is in two requests, none outside is touched."""
    T, n = 40, 3
    base, x, a, b, scale = _inputs(T, n, 16, 64, 32, F32, F32)
    _check(base, x, a, b, np.arange(len(bounds) - 1) % n, bounds, scale)


@pytest.mark.parametrize("S", [257, 1500, 5000])
def test_many_requests(S):
    """More requests than a workgroup has threads, of 0 to 40 rows."""
    rng = np.random.default_rng(S)
    size = rng.choice([0, 1, 1, 2, 3, 17, 40], S)
    bounds = np.concatenate([[0], np.cumsum(size)])
    T, n = int(bounds[-1]) + 3, 6
    base, x, a, b, scale = _inputs(T, n, 8, 32, 16, BF16, BF16)
    _check(base, x, a, b, rng.integers(-1, n, S), bounds, scale)


def test_adapter_ids_far_out_of_range():
    base, x, a, b, scale = _inputs(6, 2, 16, 64, 32, BF16, F32)
    _check(base, x, a, b, np.array([2 ** 31 - 1, -2 ** 31, 1, -1, 2, 0]), None, scale)


def test_no_scale_is_ones():
    bf = _bf()
    base, x, a, b, scale = _inputs(40, 3, 16, 128, 64, BF16, F32)
    who = _i32(np.arange(40) % 3)
    assert torch.equal(bf.lora(base, x, a, b, who), bf.lora(base, x, a, b, who, scale=torch.ones_like(scale)))


def test_no_rows():
    bf = _bf()
    base, x, a, b, _ = _inputs(0, 2, 16, 64, 32, BF16, F32)
    assert bf.lora(base, x, a, b, _i32([])).shape == (0, 32)
    assert bf.lora(base, x, a, b, _i32([1]), seq_offsets=_i32([0, 0])).shape == (0, 32)


def test_a_smaller_rank_is_padded_with_zeros():
    bf = _bf()
    base, x, a, b, scale = _inputs(50, 3, 16, 128, 64, F32, F32)
    a32 = torch.cat([a, torch.zeros_like(a)], 1).contiguous()
    b32 = torch.cat([b, torch.zeros_like(b)], 2).contiguous()
    who = _i32(np.arange(50) % 3)
    r = ol.lora(_np(base), _np(x), _np(a), _np(b), np.arange(50) % 3, None, _np(scale))
    y = bf.lora(base, x, a32, b32, who, scale=scale)
    assert (np.abs(_np(y) - r["y"]) <= _bound(r, 128, 32, F32)).all()


@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("special", [float("inf"), float("nan")])
def test_special_values_stay_in_their_row(special, xt):
    """A row with an infinity or NaN spoils its own results and no other row's."""
    bf = _bf()
    base, x, a, b, scale = _inputs(40, 2, 16, 64, 32, xt, F32)
    who = _i32(np.arange(40) // 20 % 2)
    seq = _i32([0, 20, 40])
    good = bf.lora(base, x, a, b, who[::20].contiguous(), seq_offsets=seq, scale=scale)
    x[7, 13] = special
    bad = bf.lora(base, x, a, b, who[::20].contiguous(), seq_offsets=seq, scale=scale)
    keep = torch.arange(40, device=x.device) != 7
    assert torch.equal(good[keep], bad[keep])
    assert not torch.isfinite(bad[7]).any()


@pytest.mark.parametrize("scale", [1e-30, 1e30])
def test_large_and_small_values(scale):
    """fp32 x far from 1: products of its parts neither overflow nor vanish."""
    bf = _bf()
    base, x, a, b, f = _inputs(20, 2, 16, 64, 32, F32, F32)
    x, base = x * scale, base * scale
    who = np.arange(20) % 2
    y = bf.lora(base, x, a, b, _i32(who), scale=f)
    r = ol.lora(_np(base), _np(x), _np(a), _np(b), who, None, _np(f))
    assert (np.abs(_np(y) - r["y"]) <= _bound(r, 64, 16, F32)).all()


def test_a_row_has_the_same_bits_alone():
    """What other rows and requests there are does not change a row."""
    bf = _bf()
    for xt, yt in TYPES:
        base, x, a, b, scale = _inputs(200, 5, 16, 512, 96, xt, yt)
        seq = np.array([0, 30, 31, 32, 100, 200])
        who = np.array([2, 0, 4, 1, 3])
        y = bf.lora(base, x, a, b, _i32(who), seq_offsets=_i32(seq), scale=scale)
        of = np.repeat(who, np.diff(seq))
        each = bf.lora(base, x, a, b, _i32(of), scale=scale)
        assert torch.equal(y, each)
        for t in (0, 30, 99, 199):
            one = bf.lora(base[t:t + 1].clone(), x[t:t + 1].clone(), a, b, _i32(of[t:t + 1]), scale=scale)
            assert torch.equal(one[0], y[t])


def test_far_adapters():
    """Adapters whose byte offsets pass 2^32 on both sides."""
    bf = _bf()
    dev = need_gpu()
    n, rank, d = 1024, 128, 16384
    a = torch.zeros((n, rank, d), dtype=BF16, device=dev)
    b = torch.zeros((n, d, rank), dtype=BF16, device=dev)
    base, x, al, bl, _ = _inputs(3, 1, rank, d, d, BF16, F32)
    a[-1], b[-1] = al[0], bl[0]
    a[0], b[0] = al[0], -bl[0]
    y = bf.lora(base, x, a, b, _i32([n - 1, 0, 5]))
    for t, sign in ((0, 1.0), (1, -1.0), (2, 0.0)):
        r = ol.lora(_np(base)[t:t + 1], _np(x)[t:t + 1], _np(al), sign * _np(bl), [0], None, None)
        assert (np.abs(_np(y)[t:t + 1] - r["y"]) <= _bound(r, d, rank, F32)).all()


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("rank,d_in,d_out", [(8, 96, 80), (24, 64, 64), (64, 512, 144), (72, 160, 96), (128, 288, 336)])
def test_many_rows(rank, d_in, d_out, types):
    """1,024 rows and more take two launches: bounds that leave rows out at both
    ends, requests without rows and without an adapter, tiles that end inside a
    request, neighbouring tiles of several adapters; and the bits that each
    request has alone, in one launch."""
    bf = _bf()
    T, n = 1300, 4
    base, x, a, b, scale = _inputs(T, n, rank, d_in, d_out, *types)
    seq = np.array([5, 105, 105, 110, 141, 173, 174, 500, 700, 1023, 1024, 1290])
    who = np.array([1, 0, 3, -1, 2, 0, 0, 1, n, 3, 2])
    y = _check(base, x, a, b, who, seq, scale)
    for s in range(len(who)):
        r0, r1 = seq[s], seq[s + 1]
        if r1 > r0:
            one = bf.lora(base[r0:r1].clone(), x[r0:r1].clone(), a, b, _i32(who[s:s + 1]), seq_offsets=_i32([0, r1 - r0]),
                          scale=scale)
            assert torch.equal(one, y[r0:r1]), s


def test_many_rows_of_one_request():
    base, x, a, b, scale = _inputs(5000, 2, 16, 64, 48, BF16, BF16)
    _check(base, x, a, b, np.array([1]), [0, 5000], scale)
    _check(base, x, a, b, np.array([7]), [0, 5000], scale)
    _check(base, x, a, b, np.array([0, 1]), [4999, 5000, 5000], scale)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("T,n", [(127, 5), (128, 5), (1024, 1), (1024, 40), (1500, 3), (4096, 200), (4097, 3)])
def test_many_single_rows(T, n, types):
    """Where requests outnumber the adapters, rows of one adapter share a workgroup,
    wherever they lie; rows without one among them; and the same with bounds between
    all rows."""
    bf = _bf()
    base, x, a, b, scale = _inputs(T, n, 24, 96, 48, *types)
    who = np.random.default_rng(T + n).integers(-1, n + 1, T)
    who[:40] = np.where(np.arange(40) % 3, 0, -1)
    y = _check(base, x, a, b, who, None, scale)
    assert torch.equal(bf.lora(base, x, a, b, _i32(who), seq_offsets=_i32(np.arange(T + 1)), scale=scale), y)


@pytest.mark.parametrize("T,n,d_in", [(65536, 5, 32), (65536, 1024, 64), (8000, 1024, 16384), (65536, 2, 16384)])
def test_the_most_single_rows(T, n, d_in):
    """Up to the most rows, adapters and row bytes: the bits that bounds give."""
    bf = _bf()
    dev = need_gpu()
    g = torch.Generator(device=dev).manual_seed(T + n)
    x = torch.randn((T, d_in), generator=g, device=dev)
    base = torch.randn((T, 16), generator=g, device=dev)
    a = (torch.randn((n, 8, d_in), generator=g, device=dev) / d_in ** 0.5).bfloat16()
    b = torch.randn((n, 16, 8), generator=g, device=dev).bfloat16()
    who = torch.randint(-1, n + 1, (T,), generator=g, device=dev).int()
    y = bf.lora(base, x, a, b, who)
    assert torch.equal(bf.lora(base, x, a, b, who, seq_offsets=_i32(np.arange(T + 1))), y)
    none = (who < 0) | (who >= n)
    assert torch.equal(y[none], base[none]) and not torch.equal(y[~none], base[~none])
    some = torch.randint(0, T, (40,), generator=g, device=dev).tolist() + [0, T - 1]
    r = ol.lora(_np(base[some]), _np(x[some]), _np(a), _np(b), who[some].cpu().numpy())
    assert (np.abs(_np(y[some]) - r["y"]) <= _bound(r, d_in, 8, F32)).all()


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("S,T", [(70, 150), (200, 900), (400, 1100), (900, 3000), (6000, 20000)])
def test_many_short_requests_with_bounds_out_of_order(S, T, types):
    """Gathered rows of requests of 0 to many rows, bounds that step back or leave
    the range, rows of no request between them; and the bits that rows have alone."""
    bf = _bf()
    n = 4
    base, x, a, b, scale = _inputs(T, n, 16, 64, 48, *types)
    rng = np.random.default_rng(S)
    bounds = np.sort(rng.integers(3, T - 2, S + 1))
    at = rng.integers(0, S + 1, S // 10)
    bounds[at] = rng.choice([-2 ** 31, -1, 0, T // 3, T - 5], len(at))
    if S > 300:
        bounds[-1] = 2 ** 31 - 1
    who = rng.integers(-1, n + 1, S)
    y = _check(base, x, a, b, who, bounds, scale)
    of = ol.requests_of(T, bounds)
    for t in rng.choice(np.flatnonzero(of >= 0), 5):
        one = bf.lora(base[t:t + 1].clone(), x[t:t + 1].clone(), a, b, _i32(who[of[t]:of[t] + 1]), scale=scale)
        assert torch.equal(one[0], y[t])


def test_gathered_rows_of_one_long_and_many_short_requests():
    """Rows of one adapter from a request of 700 rows and 150 single ones."""
    bf = _bf()
    base, x, a, b, scale = _inputs(850, 2, 40, 96, 64, BF16, F32)
    bounds = np.concatenate([np.arange(76), [775], 776 + np.arange(75)])
    who = np.where(np.arange(len(bounds) - 1) % 3, 1, 0)
    y = _check(base, x, a, b, who, bounds, scale)
    one = bf.lora(base[75:775].clone(), x[75:775].clone(), a, b, _i32(who[75:76]), seq_offsets=_i32([0, 700]), scale=scale)
    assert torch.equal(one, y[75:775])


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("rank,d_in,d_out", [(8, 96, 80), (40, 160, 144), (72, 64, 336), (128, 288, 64)])
def test_gathered_rows_beside_a_prompt(rank, d_in, d_out, types):
    """Many rows in two launches, gathered: single rows on both sides of a prompt whose
    adapter others share, rows without one, and the result in place of base."""
    bf = _bf()
    n, singles, prompt = 5, 190, 1500
    T = 2 * singles + prompt
    base, x, a, b, scale = _inputs(T, n, rank, d_in, d_out, *types)
    bounds = np.concatenate([np.arange(singles + 1), singles + prompt + np.arange(singles + 1)])
    who = np.random.default_rng(rank).integers(-1, n + 1, len(bounds) - 1)
    who[singles] = 2
    y = _check(base, x, a, b, who, bounds, scale)
    into = base.clone()
    bf.lora(into, x, a, b, _i32(who), seq_offsets=_i32(bounds), scale=scale, y=into)
    assert torch.equal(into, y)


@pytest.mark.parametrize("T,S", [(1000, 5000), (1000, 65536), (3000, 20000), (40000, 12000), (40000, 65536)])
def test_more_requests_than_are_looked_at_at_once(T, S):
    """Gathered rows of many requests, most of them without a row where they are more
    than the rows, some bounds out of order."""
    n = 7
    base, x, a, b, scale = _inputs(T, n, 8, 32, 16, BF16, F32)
    rng = np.random.default_rng(S)
    bounds = np.sort(rng.integers(0, T + 1, S + 1))
    at = rng.integers(0, S + 1, S // 20)
    bounds[at] = rng.integers(0, T // 2, len(at))
    _check(base, x, a, b, rng.integers(-1, n + 1, S), bounds, scale)
