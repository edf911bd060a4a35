"""GPU tests of the microscaled 4-bit floats: quantization, values, the grouped
products and the decode FFN against the fp64 oracle, their refusals, and a run
of them together.

Bars.  u = 2^-24 (half a step of fp32, relative).  A product's terms are exact
in fp32 (two 2-bit significands and a power of two), so an fp32 result differs
from the exact sum by the roundings of at most K additions, each at most a
step 2u of a partial sum that the sum of the magnitudes bounds:
|y - ref| <= 2 K u mag.  A result stored in bf16 adds 2^-8 |y|, half a step.
"""
import numpy as np
import pytest
import torch

import oracle
import oracle.mxfp4 as mx
from parity import need_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_STEP = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def _bf():
    import bit_expert_ffn_top_amd as bf
    return bf


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _rand_mx(rng, *shape, lo=117, hi=128):
    """Random codes and scales of one or several matrices, with their values."""
    codes = rng.integers(0, 256, shape[:-1] + (shape[-1] // 2,), dtype=np.uint8)
    scales = rng.integers(lo, hi, shape[:-1] + (shape[-1] // 32,)).astype(np.uint8)
    return codes, scales, mx.values(codes, scales)


def _dev(codes, scales):
    dev = need_gpu()
    return _bf().Mxfp4(torch.from_numpy(codes).to(dev), torch.from_numpy(scales).to(dev))


def _i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=need_gpu())


# --- quantization ---------------------------------------------------------------


def _check_quantize(x):
    bf = _bf()
    q = bf.mxfp4_quantize(x)
    codes, scales = mx.quantize(_np(x))
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    ref = mx.values(codes, scales)
    for dt in (torch.float32, torch.bfloat16):
        v = bf.mxfp4_dequantize(q, dtype=dt)
        assert v.dtype == dt
        assert np.array_equal(_np(v), ref, equal_nan=True), dt


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 2048), (3, 96), (5, 736), (129, 64), (257, 2048), (33, 16384)])
def test_quantize(rows, cols, dtype):
    dev = need_gpu()
    g = torch.Generator().manual_seed(rows * 7 + cols)
    x = torch.randn((rows, cols), generator=g) * torch.exp(4 * torch.randn((rows, 1), generator=g))
    _check_quantize(x.to(dev).to(dtype))


def test_quantize_stack_of_matrices():
    dev = need_gpu()
    x = torch.randn((3, 5, 96), generator=torch.Generator().manual_seed(2)).to(dev)
    q = _bf().mxfp4_quantize(x)
    assert q.shape == (3, 5, 96) and q.codes.shape == (3, 5, 48) and q.scales.shape == (3, 5, 3)
    _check_quantize(x)


@pytest.mark.parametrize("e", [-149, -130, -127, -126, -125, -124, -64, -62, -61, -60, 0, 60, 125, 127])
def test_quantize_around_every_border(e):
    """Values on, just below and just above each border of the grid, blocks of
    every kind of exponent (subnormal ones, the scale's lower end, the largest
    finite values); signs and signed zeros kept."""
    dev = need_gpu()
    grid = np.array([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7, 7.99], np.float64)
    with np.errstate(under="ignore", over="ignore"):
        v = np.ldexp(grid, e - 2).astype(np.float32)
        v = np.concatenate([v, np.nextafter(v, np.float32(np.inf)), np.nextafter(v, np.float32(0)), -v])
    v = v[np.isfinite(v)]
    top = np.float32(np.ldexp(1.0, e)) if e <= 127 else np.float32(0)
    rows = []
    for i in range(0, len(v), 30):
        blk = np.zeros(32, np.float32)
        part = v[i:i + 30]
        blk[:len(part)] = part
        blk[30], blk[31] = top, -0.0
        rows.append(blk)
    _check_quantize(torch.from_numpy(np.stack(rows)).to(dev))


def test_quantize_zero_and_bad_blocks():
    dev = need_gpu()
    x = torch.randn((4, 160), generator=torch.Generator().manual_seed(3))
    x[0, :32] = 0
    x[1, 33] = float("nan")
    x[2, 70] = float("inf")
    x[2, 100] = float("-inf")
    x[3, 159] = float("nan")
    for dt in (torch.float32, torch.bfloat16):
        _check_quantize(x.to(dev).to(dt))
    q = _bf().mxfp4_quantize(x.to(dev))
    bad = (q.scales == 255).cpu()
    assert bad.sum() == 4 and bad[1, 1] and bad[2, 2] and bad[2, 3] and bad[3, 4]


def test_values_of_every_code_and_scale():
    """All 256 bytes of codes under all 256 scales; a scale of 255 is NaN."""
    dev = need_gpu()
    bf = _bf()
    codes = np.repeat(np.arange(256, dtype=np.uint8).reshape(1, 16, 16), 256, 0).reshape(256, 256)
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    q = _dev(codes, scales)
    with np.errstate(over="ignore"):
        ref = mx.values(codes, scales).astype(np.float32).astype(np.float64)
    for dt in (torch.float32, torch.bfloat16):
        got = _np(bf.mxfp4_dequantize(q, dtype=dt))
        assert np.array_equal(got, ref, equal_nan=True), dt
    del dev


# --- products -------------------------------------------------------------------


def _close(y, ref, mag, K, dtype):
    got = _np(y)
    bound = 2 * K * U * mag + HALF_STEP[dtype] * (np.abs(ref) + 2 * K * U * mag)
    err = np.abs(got - ref)
    assert (err <= bound).all(), (float((err - bound).max()), float((err / np.maximum(bound, 1e-300)).max()))


def _bounds(rng, rows, G, empty=0.3):
    """Group bounds over `rows` rows, some groups empty."""
    w = rng.random(G) * (rng.random(G) >= empty)
    if w.sum() == 0:
        w[0] = 1
    c = np.floor(np.cumsum(w) / w.sum() * rows).astype(int)
    c[-1] = rows
    return np.concatenate([[0], c])


DENSE = [  # R, N, K
    (1, 16, 32), (1, 2048, 768), (2, 48, 64), (15, 16, 96), (16, 64, 128), (17, 272, 160), (33, 80, 256),
    (63, 16, 288), (64, 128, 512), (65, 1040, 704), (130, 96, 1056), (200, 256, 2048), (257, 528, 736),
    (300, 512, 256), (511, 256, 16384),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,N,K", DENSE, ids=[f"R{c[0]}_N{c[1]}_K{c[2]}" for c in DENSE])
def test_linear_dense(R, N, K, dtype):
    rng = np.random.default_rng(R + N + K)
    ac, as_, av = _rand_mx(rng, R, K)
    wc, ws, wv = _rand_mx(rng, N, K)
    y = _bf().mxfp4_linear(_dev(ac, as_), _dev(wc, ws), dtype=dtype)
    assert y.shape == (R, N) and y.dtype == dtype
    _close(y, av @ wv.T, np.abs(av) @ np.abs(wv.T), K, dtype)


GROUPED = [  # rows of A, R, G, N, K
    (4, 9, 3, 16, 32), (37, 148, 60, 1040, 704), (64, 640, 128, 64, 96), (50, 500, 7, 144, 288),
    (40, 1300, 5, 272, 160), (700, 2000, 3, 256, 256), (10, 10, 1024, 32, 64), (300, 3000, 12, 512, 128),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,R,G,N,K", GROUPED, ids=[f"M{c[0]}_R{c[1]}_G{c[2]}_N{c[3]}_K{c[4]}" for c in GROUPED])
def test_linear_grouped(M, R, G, N, K, dtype):
    """Ragged and empty groups, gathered rows with a divisor, rows past the
    last group left as they were, rows without a source."""
    bf = _bf()
    dev = need_gpu()
    rng = np.random.default_rng(M + R + G + N + K)
    ac, as_, av = _rand_mx(rng, M, K)
    wc, ws, wv = _rand_mx(rng, G, N, K)
    used = R - 2 if R > 4 else R
    off = _bounds(rng, used, G)
    div = 3
    src = rng.integers(0, M * div, R)
    src[0], src[used // 2] = -1, M * div
    y = torch.full((R, N), 7.0, dtype=dtype, device=dev)
    bf.mxfp4_linear(_dev(ac, as_), _dev(wc, ws), _i32(off), _i32(src), div, y=y)
    ref, mag, cov = mx.product(av, wv, off, np.where(src < 0, -1, src // div))
    assert cov.sum() == used
    assert (y[used:] == 7).all()
    ref[~cov], mag[~cov] = 7.0, 0.0
    _close(y, ref, mag, K, dtype)


WIDE = [  # enough row tiles and columns for the kernel of full tiles: M, R, G, N, K
    (40, 1300, 600, 272, 160), (50, 900, 512, 528, 288), (31, 700, 530, 512, 640), (64, 640, 640, 400, 704),
    (9, 1200, 520, 256, 1280), (77, 5000, 300, 512, 256), (200, 3000, 3, 8448, 64), (1300, 1300, 1, 12032, 96),
    (1000, 1000, 2, 16640, 512), (20, 530, 530, 256, 2304),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,R,G,N,K", WIDE, ids=[f"M{c[0]}_R{c[1]}_G{c[2]}_N{c[3]}_K{c[4]}" for c in WIDE])
def test_wide_products(M, R, G, N, K, dtype):
    """Groups of one row and of thousands, several tiles to a group, a last
    step and a last chunk of scales that a row ends inside; both products."""
    _check_products(M, R, G, N, K, dtype)


FEW = [  # too little work for that kernel: one to over 64 rows a group, rows of up to 64 chunks
    (30, 100, 40, 512, 1312), (50, 900, 40, 512, 2400), (60, 1500, 40, 448, 1056), (16, 40, 40, 448, 4128),
    (20, 60, 6, 64, 4384), (20, 300, 3, 80, 8448), (9, 33, 1, 32, 16384), (70, 65, 1, 64, 5024),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,R,G,N,K", FEW, ids=[f"M{c[0]}_R{c[1]}_G{c[2]}_N{c[3]}_K{c[4]}" for c in FEW])
def test_products_of_few_rows(M, R, G, N, K, dtype):
    """One, two and four token tiles, a tile that shares its group with others,
    more chunks than are asked for ahead, rows that end inside one."""
    _check_products(M, R, G, N, K, dtype)


def _check_products(M, R, G, N, K, dtype):
    bf = _bf()
    dev = need_gpu()
    rng = np.random.default_rng(M + R + G + N + K)
    ac, as_, av = _rand_mx(rng, M, K, lo=122, hi=127)
    wc, ws, wv = _rand_mx(rng, G, N, K, lo=118, hi=123)
    used = R - 3
    off = _bounds(rng, used, G)
    src = rng.integers(0, 2 * M, R)
    src[1], src[used - 1] = -1, 2 * M
    gather = (_i32(off), _i32(src), 2)
    ref, mag, cov = mx.product(av, wv, off, np.where(src < 0, -1, src // 2))
    y = torch.full((R, N), 7.0, dtype=dtype, device=dev)
    bf.mxfp4_linear(_dev(ac, as_), _dev(wc, ws), *gather, y=y)
    assert (y[used:] == 7).all() and not cov[used:].any()
    _close(y[:used], ref[:used], mag[:used], K, dtype)
    h = torch.full((R, N // 2), 7.0, dtype=dtype, device=dev)
    if N % 64 == 0:
        bf.mxfp4_gate_up(_dev(ac, as_), _dev(wc, ws), *gather, h=h)
        g, u, d = ref[:used, 0::2], ref[:used, 1::2], 2 * K * U * mag[:used]
        want = mx.silu(g) * u
        bound = _silu_bound(g, u, d[:, 0::2], d[:, 1::2])
        bound += HALF_STEP[dtype] * (np.abs(want) + bound) + 1e-40
        assert (np.abs(_np(h[:used]) - want) <= bound).all()
        assert (h[used:] == 7).all()


def _silu_bound(g, u, dg, du):
    """|silu(g') u' - silu(g) u| for g', u' off by dg, du: |silu'| <= 1.1 and
    |silu(z)| <= |z|; the function itself and the product in fp32 add 8 u."""
    h = np.abs(mx.silu(g)) + 1.1 * dg
    return 1.1 * dg * (np.abs(u) + du) + np.abs(mx.silu(g)) * du + 8 * U * h * (np.abs(u) + du)


GATE_UP = [  # M, R, G, F, K
    (1, 1, 1, 32, 32), (5, 11, 2, 64, 96), (64, 640, 96, 96, 160), (30, 900, 4, 128, 288),
    (600, 1500, 5, 160, 256), (64, 64, 64, 768, 2048),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,R,G,F,K", GATE_UP, ids=[f"M{c[0]}_R{c[1]}_G{c[2]}_F{c[3]}_K{c[4]}" for c in GATE_UP])
def test_gate_up(M, R, G, F, K, dtype):
    bf = _bf()
    dev = need_gpu()
    rng = np.random.default_rng(M + R + G + F + K)
    ac, as_, av = _rand_mx(rng, M, K, lo=122, hi=127)
    wc, ws, wv = _rand_mx(rng, G, 2 * F, K, lo=118, hi=123)
    off = _bounds(rng, R, G)
    src = rng.integers(0, M, R)
    h = torch.full((R, F), 7.0, dtype=dtype, device=dev)
    bf.mxfp4_gate_up(_dev(ac, as_), _dev(wc, ws), _i32(off), _i32(src), 1, h=h)
    p, mag, cov = mx.product(av, wv, off, src)
    assert cov.all()
    g, u = p[:, 0::2], p[:, 1::2]
    d = 2 * K * U * mag
    ref = mx.silu(g) * u
    bound = _silu_bound(g, u, d[:, 0::2], d[:, 1::2])
    bound += HALF_STEP[dtype] * (np.abs(ref) + bound)
    err = np.abs(_np(h) - ref)
    assert (err <= bound).all(), float((err / np.maximum(bound, 1e-300)).max())


def test_products_of_extreme_scales():
    """Scales at both ends: an fp32 result overflows to infinity or stays
    exact, and a NaN block reaches only the rows that read it."""
    bf = _bf()
    rng = np.random.default_rng(5)
    K, N, R = 256, 32, 40
    ac, as_, _ = _rand_mx(rng, R, K)
    wc, ws, _ = _rand_mx(rng, N, K)
    as_[3, 2], ws[7, 5] = 255, 255
    as_[4], as_[5] = 0, 250
    ws[9], ws[10] = 252, 1
    y = _np(bf.mxfp4_linear(_dev(ac, as_), _dev(wc, ws)))
    ac0, ws0 = np.where(as_ == 255, 127, as_), np.where(ws == 255, 127, ws)
    av, wv = mx.values(ac, ac0), mx.values(wc, ws0)
    ref, mag = av @ wv.T, np.abs(av) @ np.abs(wv.T)
    nan = np.zeros((R, N), bool)
    nan[3], nan[:, 7] = True, True
    assert np.array_equal(np.isnan(y), nan)
    big = mag > 1e38                                  # the fp32 sum may pass the largest value
    small = ~nan & ~big
    # products below the smallest normal number may lose bits: 2^-126 each
    assert (np.abs(y - ref)[small] <= (2 * K * U * mag + K * 2.0 ** -126)[small]).all()
    assert big.any() and not np.isnan(y[big & ~nan]).any()


def test_rows_do_not_depend_on_the_batch():
    """A call repeated gives the same bits; a row alone, among few and among
    many rows differs by no more than the order of its sum."""
    bf = _bf()
    rng = np.random.default_rng(6)
    R, N, K = 600, 272, 416
    ac, as_, _ = _rand_mx(rng, R, K)
    wc, ws, _ = _rand_mx(rng, N, K)
    W = _dev(wc, ws)
    full = bf.mxfp4_linear(_dev(ac, as_), W)
    again = bf.mxfp4_linear(_dev(ac, as_), W)
    assert torch.equal(full, again)
    for lo, hi in ((0, 1), (599, 600), (17, 20), (100, 140), (3, 300)):
        part = bf.mxfp4_linear(_dev(ac[lo:hi].copy(), as_[lo:hi].copy()), W)
        assert torch.allclose(part, full[lo:hi], rtol=0, atol=float(2 * K * U * 36 * K)), (lo, hi)


def test_descending_and_outside_bounds_are_clamped():
    """Bounds that are not ascending or lie outside the rows touch no other
    memory: groups of negative length are empty, bounds are clamped."""
    bf = _bf()
    dev = need_gpu()
    rng = np.random.default_rng(8)
    R, G, N, K = 20, 4, 32, 64
    ac, as_, av = _rand_mx(rng, R, K)
    wc, ws, wv = _rand_mx(rng, G, N, K)
    y = torch.full((R + 8, N), 7.0, device=dev)
    bf.mxfp4_linear(_dev(ac, as_), _dev(wc, ws), _i32([-5, 6, 4, 12, 1 << 30]), y=y[:R])
    ref, mag, _ = mx.product(av, wv, [0, 6, 6, 12, R])
    # group 1 is empty, group 2 starts at its own bound: rows 4..11 are its
    ref2, _, _ = mx.product(av, wv, [0, 4, 4, 12, R])
    got = _np(y[:R])
    for r in range(R):
        ok = [np.abs(got[r] - q[r]).max() <= (2 * K * U * mag[r]).max() for q in (ref, ref2)]
        assert any(ok), r
    assert (y[R:] == 7).all()


@pytest.mark.parametrize("G,R,N,K", [(4, 20, 32, 64), (700, 900, 272, 96), (1024, 3000, 512, 64)])
def test_descending_bounds_put_no_row_in_two_groups(G, R, N, K):
    """Bounds in any order: one below an earlier one counts as that one, so
    the result is that of their running maximum, with the same bits each time."""
    bf = _bf()
    dev = need_gpu()
    rng = np.random.default_rng(G + R)
    ac, as_, _ = _rand_mx(rng, R, K)
    wc, ws, _ = _rand_mx(rng, G, N, K)
    A, W = _dev(ac, as_), _dev(wc, ws)
    off = np.sort(rng.integers(0, R, G + 1))
    off[rng.integers(0, G + 1, G // 3 + 1)] = rng.integers(-9, R + 9, G // 3 + 1)
    top = np.maximum.accumulate(np.clip(off, 0, R))
    want = torch.full((R, N), 7.0, device=dev)
    bf.mxfp4_linear(A, W, _i32(top), y=want)
    for _ in range(3):
        y = torch.full((R, N), 7.0, device=dev)
        bf.mxfp4_linear(A, W, _i32(off), y=y)
        assert torch.equal(y, want)


def test_no_rows():
    bf = _bf()
    dev = need_gpu()
    rng = np.random.default_rng(9)
    wc, ws, _ = _rand_mx(rng, 2, 64, 64)
    ac, as_, _ = _rand_mx(rng, 3, 64)
    assert bf.mxfp4_linear(_dev(ac, as_), _dev(wc, ws), _i32([0, 0, 0]), _i32([])).shape == (0, 64)
    y = torch.full((3, 64), 7.0, device=dev)
    bf.mxfp4_linear(_dev(ac, as_), _dev(wc, ws), _i32([0, 0, 0]), y=y)      # every group empty
    assert (y == 7).all()
    assert bf.mxfp4_quantize(torch.empty((0, 64), device=dev)).codes.shape == (0, 32)


def test_more_than_2_31_outputs():
    """Rows past 2^31 outputs (and past 2^32 bytes) land where they belong."""
    bf = _bf()
    dev = need_gpu()
    rng = np.random.default_rng(10)
    R, N, K = 1_100_000, 2048, 32
    wc, ws, wv = _rand_mx(rng, N, K)
    ac, as_, av = _rand_mx(rng, 64, K)
    A, W = _dev(ac, as_), _dev(wc, ws)
    src = torch.arange(R, dtype=torch.int32, device=dev) % 64
    y = bf.mxfp4_linear(A, W, None, src)
    ref = torch.from_numpy((av @ wv.T).astype(np.float32)).to(dev)
    bound = float(2 * K * U * (np.abs(av) @ np.abs(wv.T)).max())
    for lo in (0, R // 2, R - 4096):
        want = ref[src[lo:lo + 4096].long()]
        assert (y[lo:lo + 4096] - want).abs().max() <= bound, lo
    del y
    x = torch.zeros((R, 2048), dtype=torch.bfloat16, device=dev)
    x[-1, -40:] = 3.0
    q = bf.mxfp4_quantize(x)
    assert (q.scales[-1, -1] == 126) and not q.codes[:-1].any()
    assert (bf.mxfp4_dequantize(q, dtype=torch.bfloat16)[-1, -40:] == 3).all()


# --- decode FFN -----------------------------------------------------------------

DECODE = [  # T, k, n, d, F, shared
    (1, 10, 16, 2048, 768, True), (4, 10, 40, 2048, 768, True), (1, 1, 1, 32, 32, False),
    (2, 3, 5, 96, 64, True), (3, 21, 30, 544, 160, False), (4, 16, 20, 1056, 1056, True),
    (1, 64, 70, 64, 4096, False), (1, 2, 3, 4096, 544, True), (2, 0, 2, 128, 96, True), (1, 7, 9, 736, 512, True),
]


def _decode_case(T, k, n, d, F, shared, seed=0):
    rng = np.random.default_rng(T + k + n + d + F + seed)
    gc, gs, gv = _rand_mx(rng, n, 2 * F, d, lo=117, hi=121)
    dc, ds, dv = _rand_mx(rng, n, d, F, lo=118, hi=122)
    x = rng.normal(size=(T, d)).astype(np.float32)
    slot = np.stack([rng.permutation(n)[:k] if k <= n else rng.integers(0, n, k) for _ in range(T)]) \
        if k else np.zeros((T, 0), int)
    w = rng.random((T, k)).astype(np.float32)
    return (gc, gs, gv), (dc, ds, dv), x, slot.astype(np.int32), w, (n - 1 if shared else -1)


def _check_decode(y, gv, dv, x, slot, w, shared):
    """Bar: dot products of d and F fp32 multiply-adds (each rounding at most
    u of a partial sum of magnitudes), silu as above, then the weighted sum."""
    xd = x.astype(np.float64)
    n, F2, d = gv.shape
    ref = mx.ffn_decode(xd, gv, dv, slot, w.astype(np.float64), shared)
    bound = np.abs(xd).copy()
    for t in range(x.shape[0]):
        tot = np.abs(xd[t]).copy()
        err = np.zeros(d)
        for i in range(slot.shape[1] + 1):
            m, wt = (shared, 1.0) if i == slot.shape[1] else (slot[t, i], float(w[t, i]))
            if not 0 <= m < n:
                continue
            p, pm = gv[m] @ xd[t], np.abs(gv[m]) @ np.abs(xd[t])
            g, u, dp = p[0::2], p[1::2], (d + 8) * U * pm
            h, dh = np.abs(mx.silu(g) * u), _silu_bound(g, u, dp[0::2], dp[1::2])
            o = np.abs(dv[m]) @ (h + dh)
            err += wt * (np.abs(dv[m]) @ dh + (F2 // 2 + 8) * U * o)
            tot += wt * o
        bound[t] = err + (slot.shape[1] + 8) * U * tot
    e = np.abs(_np(y) - ref)
    assert (e <= bound).all(), float((e / bound).max())


@pytest.mark.parametrize("case", DECODE, ids=["T%d_k%d_n%d_d%d_F%d_s%d" % c for c in DECODE])
def test_ffn_decode(case):
    bf = _bf()
    (gc, gs, gv), (dc, ds, dv), x, slot, w, shared = _decode_case(*case)
    dev = need_gpu()
    args = (_dev(gc, gs), _dev(dc, ds), torch.from_numpy(x).to(dev), _i32(slot).reshape(slot.shape),
            torch.from_numpy(w).to(dev))
    y = bf.mxfp4_ffn_decode(*args, shared_slot=shared)
    assert torch.equal(y, bf.mxfp4_ffn_decode(*args, shared_slot=shared))
    _check_decode(y, gv, dv, x, slot, w, shared)


def test_ffn_decode_slots_outside_the_pool():
    """Negative slots and slots at or past the pool add nothing (and read
    nothing); a token whose every slot is outside gives x."""
    bf = _bf()
    dev = need_gpu()
    (gc, gs, gv), (dc, ds, dv), x, slot, w, _ = _decode_case(3, 5, 6, 128, 96, False)
    slot[0, 1], slot[0, 3], slot[2] = -1, 6, [6, 1 << 30, -5, -1, 7]
    y = bf.mxfp4_ffn_decode(_dev(gc, gs), _dev(dc, ds), torch.from_numpy(x).to(dev), _i32(slot),
                            torch.from_numpy(w).to(dev))
    _check_decode(y, gv, dv, x, slot, w, -1)
    assert np.array_equal(_np(y)[2], x[2].astype(np.float64))


def test_ffn_decode_token_alone_and_among_others():
    """A verified token has the bits it has alone, also where the tokens share
    experts (every token the same ones, some in another order)."""
    bf = _bf()
    dev = need_gpu()
    (gc, gs, _), (dc, ds, _), x, slot, w, shared = _decode_case(4, 6, 12, 2048, 768, True)
    slot[1] = slot[0]
    slot[2] = slot[0][::-1]
    slot[3, :3] = slot[0, :3]
    G, D = _dev(gc, gs), _dev(dc, ds)
    xs, sl, ws = torch.from_numpy(x).to(dev), _i32(slot), torch.from_numpy(w).to(dev)
    for T in (2, 3, 4):
        y = bf.mxfp4_ffn_decode(G, D, xs[:T].contiguous(), sl[:T].contiguous(), ws[:T].contiguous(),
                                shared_slot=shared)
        for t in range(T):
            one = bf.mxfp4_ffn_decode(G, D, xs[t:t + 1].clone(), sl[t:t + 1].clone(), ws[t:t + 1].clone(),
                                      shared_slot=shared)
            assert torch.equal(y[t], one[0]), (T, t)


def test_ffn_decode_same_expert_twice():
    bf = _bf()
    dev = need_gpu()
    (gc, gs, gv), (dc, ds, dv), x, slot, w, shared = _decode_case(2, 4, 5, 96, 64, True)
    slot[0] = 2
    slot[1, 3] = shared
    y = bf.mxfp4_ffn_decode(_dev(gc, gs), _dev(dc, ds), torch.from_numpy(x).to(dev), _i32(slot),
                            torch.from_numpy(w).to(dev), shared_slot=shared)
    _check_decode(y, gv, dv, x, slot, w, shared)


# --- grouping, and the whole layer ----------------------------------------------


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (3, 4, 7), (100, 10, 512), (65, 64, 64), (1000, 3, 1024)])
def test_group_pairs(T, k, E):
    rng = np.random.default_rng(T + k + E)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    idx[T // 2, k // 2] = -1
    idx[T - 1, 0] = E
    off, pos, rows = (t.cpu().numpy() for t in _bf().group_pairs(_i32(idx), E))
    woff, wpos, wrows = mx.group_pairs(idx, E)
    assert np.array_equal(off, woff) and np.array_equal(pos, wpos)
    assert np.array_equal(rows[:len(wrows)], wrows)


def _layer(T, E, k, d, F, seed, dev):
    g = torch.Generator(device=dev).manual_seed(seed)
    bf = _bf()
    gu = bf.mxfp4_quantize(torch.randn((E, 2 * F, d), generator=g, device=dev) / d ** 0.5)
    dn = bf.mxfp4_quantize(torch.randn((E, d, F), generator=g, device=dev) / F ** 0.5)
    x = torch.randn((T, d), generator=g, device=dev)
    logits = torch.randn((T, E), generator=g, device=dev)
    return gu, dn, x, logits


def test_prefill_layer_over_4bit_experts():
    """route_topk -> group_pairs -> quantize -> gate_up -> quantize -> linear ->
    combine, every stage against the oracle on the stage before's own output
    (4-bit codes of a sum next to a border may differ, so no error may be
    carried over them)."""
    bf = _bf()
    dev = need_gpu()
    T, E, k, d, F = 203, 24, 5, 256, 96
    gu, dn, x, logits = _layer(T, E, k, d, F, 11, dev)
    idx, w = bf.route_topk(logits, k)
    off, pos, rows = bf.group_pairs(idx, E)
    xq = bf.mxfp4_quantize(x)
    h = bf.mxfp4_gate_up(xq, gu, off, rows, k)
    hq = bf.mxfp4_quantize(h)
    y = bf.mxfp4_linear(hq, dn, off)
    out = bf.combine(x, y, pos, w)
    torch.cuda.synchronize()
    ridx, rw = oracle.route_topk(logits.cpu().numpy(), k)
    assert np.array_equal(idx.cpu().numpy(), ridx)
    woff, wpos, wrows = mx.group_pairs(ridx, E)
    assert np.array_equal(off.cpu().numpy(), woff) and np.array_equal(pos.cpu().numpy(), wpos)
    gv, dv = (mx.values(q.codes.cpu().numpy(), q.scales.cpu().numpy()) for q in (gu, dn))
    xc, xs = mx.quantize(_np(x))
    assert np.array_equal(xq.codes.cpu().numpy(), xc) and np.array_equal(xq.scales.cpu().numpy(), xs)
    p, mag, _ = mx.product(mx.values(xc, xs), gv, woff, wrows // k)
    g, u, dd = p[:, 0::2], p[:, 1::2], 2 * d * U * mag
    ref = mx.silu(g) * u
    b = _silu_bound(g, u, dd[:, 0::2], dd[:, 1::2])
    assert (np.abs(_np(h) - ref) <= b + 2.0 ** -8 * (np.abs(ref) + b)).all()
    hc, hs = mx.quantize(_np(h))
    assert np.array_equal(hq.codes.cpu().numpy(), hc) and np.array_equal(hq.scales.cpu().numpy(), hs)
    yr, ymag, _ = mx.product(mx.values(hc, hs), dv, woff)
    _close(y, yr, ymag, F, torch.float32)
    yy = _np(y)
    full = _np(x) + (rw[:, :, None] * yy[wpos]).sum(1)
    tol = (k + 2) * U * (np.abs(_np(x)) + (rw[:, :, None] * np.abs(yy[wpos])).sum(1)) + 1e-6 * np.abs(full)
    assert (np.abs(_np(out) - full) <= tol + 1e-6 * (rw[:, :, None] * np.abs(yy[wpos])).sum(1)).all()


def test_decode_layer_over_4bit_experts():
    """route_topk -> cache_lookup -> ffn_decode with some experts not cached."""
    bf = _bf()
    dev = need_gpu()
    T, E, k, d, F = 4, 20, 6, 256, 128
    gu, dn, x, logits = _layer(T, E, k, d, F, 12, dev)
    idx, w = bf.route_topk(logits, k)
    table = torch.arange(E, dtype=torch.int32, device=dev)
    table[::4] = -1
    slot, _, _, n_miss = bf.cache_lookup(idx, table)
    y = bf.mxfp4_ffn_decode(gu, dn, x, slot, w, shared_slot=E - 1)
    assert int(n_miss[1]) > 0
    gv, dv = (mx.values(q.codes.cpu().numpy(), q.scales.cpu().numpy()) for q in (gu, dn))
    _check_decode(y, gv, dv, x.cpu().numpy(), slot.cpu().numpy(), w.cpu().numpy(), E - 1)


# --- streams, graphs, refusals ---------------------------------------------------


def test_streams_and_graphs():
    """The layer on a side stream, and captured in a graph that is replayed
    with other inputs between eager calls: always the eager bits."""
    bf = _bf()
    dev = need_gpu()
    T, E, k, d, F = 4, 16, 4, 256, 64
    gu, dn, x, logits = _layer(T, E, k, d, F, 13, dev)
    xs = [x, torch.flip(x, [0]) * 1.5, x * 0.25]
    lgs = [logits, torch.flip(logits, [1]), -logits]

    def step(x, lg):
        idx, w = bf.route_topk(lg, k)
        off, pos, rows = bf.group_pairs(idx, E)
        h = bf.mxfp4_gate_up(bf.mxfp4_quantize(x), gu, off, rows, k)
        y = bf.mxfp4_linear(bf.mxfp4_quantize(h), dn, off)
        return bf.combine(x, y, pos, w), bf.mxfp4_ffn_decode(gu, dn, x, idx, w, shared_slot=3)

    eager = [step(a, b) for a, b in zip(xs, lgs)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q = bf.mxfp4_quantize(x, stream=side)
    one = bf.mxfp4_ffn_decode(gu, dn, x, bf_idx := bf.route_topk(logits, k)[0], bf.route_topk(logits, k)[1],
                              shared_slot=3)
    side.wait_stream(torch.cuda.current_stream())
    idx, w = bf.route_topk(logits, k)
    torch.cuda.synchronize()
    two = bf.mxfp4_ffn_decode(gu, dn, x, idx, w, shared_slot=3, stream=side)
    off, pos, rows = bf.group_pairs(idx, E, stream=side)
    h = bf.mxfp4_gate_up(q, gu, off, rows, k, stream=side)
    y = bf.mxfp4_linear(bf.mxfp4_quantize(h, stream=side), dn, off, stream=side)
    v = bf.mxfp4_dequantize(q, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(one, eager[0][1]) and torch.equal(two, eager[0][1]) and torch.equal(bf_idx, idx)
    assert torch.equal(bf.combine(x, y, pos, w), eager[0][0])
    assert torch.equal(v, bf.mxfp4_dequantize(bf.mxfp4_quantize(x)))
    sx, sl = x.clone(), logits.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(sx, sl)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(sx, sl)
    for i in (1, 2, 0, 1, 2):
        sx.copy_(xs[i])
        sl.copy_(lgs[i])
        graph.replay()
        torch.cuda.synchronize()
        again = step(xs[i], lgs[i])
        for a, b, c in zip(got, eager[i], again):
            assert torch.equal(a, b) and torch.equal(c, b), i


def test_device_refusals():
    bf = _bf()
    dev = need_gpu()
    x = torch.randn((4, 64), device=dev)
    with pytest.raises(ValueError, match="contiguous"):
        bf.mxfp4_quantize(x.t().contiguous().t())
    q = bf.mxfp4_quantize(x)
    with pytest.raises(ValueError, match="must be a device tensor"):
        bf.mxfp4_dequantize(bf.Mxfp4(q.codes, q.scales.cpu()))
    w = bf.mxfp4_quantize(torch.randn((40, 64), device=dev))
    with pytest.raises(bf.MoeError, match="invalid argument"):      # 40 rows: no multiple of 16
        bf.mxfp4_linear(q, w)
    with pytest.raises(bf.MoeError, match="misaligned"):
        buf = torch.empty((4 * 64 + 4,), device=dev)
        bf.mxfp4_dequantize(q, y=buf[1:257].view(4, 64))
    ws = torch.empty((64,), dtype=torch.uint8, device=dev)
    gu = bf.mxfp4_quantize(torch.randn((2, 64, 64), device=dev))
    dn = bf.mxfp4_quantize(torch.randn((2, 64, 32), device=dev))
    sl = torch.zeros((4, 1), dtype=torch.int32, device=dev)
    with pytest.raises(bf.MoeError, match="workspace"):
        bf.mxfp4_ffn_decode(gu, dn, x, sl, torch.ones((4, 1), device=dev), ws=ws)
    with pytest.raises(bf.MoeError, match="invalid argument"):
        bf.mxfp4_ffn_decode(gu, dn, torch.cat([x, x]), torch.cat([sl, sl]), torch.ones((8, 1), device=dev))
