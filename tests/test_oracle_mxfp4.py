"""Pins of the 4-bit float oracle: the format's table, hand-built blocks and
brute force over every code."""
import numpy as np

import oracle.mxfp4 as mx


def test_code_values():
    assert mx.code_values().tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6]


def test_every_code_survives_requantization():
    """A block that holds every code and a 6 keeps codes and scale."""
    codes = np.array([[(2 * i % 16) | ((2 * i + 1) % 16) << 4 for i in range(16)]], np.uint8)
    for s in (0, 1, 64, 127, 200, 252):
        scales = np.array([[s]], np.uint8)
        c2, s2 = mx.quantize(mx.values(codes, scales))
        assert np.array_equal(s2, scales) and np.array_equal(c2, codes), s


def test_hand_block():
    x = np.zeros((1, 32))
    x[0, :12] = [7.9, 5.0, -5.0, 5.1, 2.5, 3.5, 0.25, 0.26, 0.75, -1.25, 1.75, -0.0]
    codes, scales = mx.quantize(x)
    assert scales.tolist() == [[127]]
    v = mx.values(codes, scales)[0]
    assert v[:12].tolist() == [6, 4, -4, 6, 2, 4, 0, 0.5, 1, -1, 2, 0]
    assert np.signbit(v[11]) and not np.signbit(v[6])


def test_scale_rule():
    for top, s in ((8.0, 128), (7.999, 127), (1.0, 125), (6.0, 127), (2.0 ** -125, 0), (2.0 ** -124, 1),
                   (2.0 ** -149, 0), (0.0, 0), (3.4e38, 252)):
        x = np.zeros((1, 32))
        x[0, 5] = top
        assert mx.quantize(x)[1].tolist() == [[s]], top
    x = np.zeros((1, 64))
    x[0, 3], x[0, 40] = np.inf, np.nan
    codes, scales = mx.quantize(x)
    assert scales.tolist() == [[255, 255]] and not codes.any() and np.isnan(mx.values(codes, scales)).all()


def test_product_and_groups():
    rng = np.random.default_rng(0)
    a, w = rng.normal(size=(5, 32)), rng.normal(size=(3, 4, 32))
    y, _, cov = mx.product(a, w, [0, 2, 2, 4], np.array([4, 0, 9, 1, 2]))
    assert cov.tolist() == [True] * 4 + [False]
    assert np.allclose(y[0], w[0] @ a[4]) and np.allclose(y[3], w[2] @ a[1]) and not y[2].any()
    idx = np.array([[2, 0], [0, 7], [1, 2]], np.int32)
    off, pos, rows = mx.group_pairs(idx, 3)
    assert off.tolist() == [0, 2, 3, 5] and rows.tolist() == [1, 2, 4, 0, 5]
    assert pos.tolist() == [[3, 0], [1, -1], [2, 4]]
