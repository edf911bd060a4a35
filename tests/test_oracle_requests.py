"""Pins of the oracles of the dispatch and back, the adapters and the verification
of drafted tokens: hand-built values, invariants, and brute-force enumeration."""
import itertools

import numpy as np

import oracle.dispatch as od
import oracle.drafts as odr
import oracle.lora as ol


def test_positions_by_hand():
    idx = np.array([[2, 0], [0, 5], [2, 2], [-1, 1]])
    offsets, pos = od.positions(idx, 3)
    assert offsets.tolist() == [0, 2, 3, 6]
    assert pos.tolist() == [[3, 0], [1, -1], [4, 5], [-1, 2]]


def test_combine_and_its_gradient_by_hand():
    rows = np.array([[1.0, 2.0], [3.0, -4.0], [10.0, 10.0]])
    pos = np.array([[1, 0], [-1, 2], [3, -1]])
    w = np.array([[2.0, 0.5], [9.0, 1.0], [1.0, 1.0]])
    y, mag = od.combine_rows(rows, pos, w, np.array([[1.0, 1.0], [0.0, -1.0], [7.0, 7.0]]))
    assert y.tolist() == [[7.5, -6.0], [10.0, 9.0], [7.0, 7.0]]
    assert mag.tolist() == [[7.5, 10.0], [10.0, 11.0], [7.0, 7.0]]
    drows, dw, mag = od.combine_backward(np.array([[1.0, 3.0], [2.0, 0.0], [5.0, 5.0]]), rows, pos, w)
    assert drows.tolist() == [[0.5, 1.5], [2.0, 6.0], [2.0, 0.0]]
    assert dw.tolist() == [[-9.0, 7.0], [0.0, 20.0], [0.0, 0.0]] and mag[0].tolist() == [15.0, 7.0]


def test_the_gradient_is_the_adjoint():
    """<dy, combine(rows, w)> = <drows, rows> = <dw, w>: linear in both."""
    rng = np.random.default_rng(1)
    idx = np.stack([rng.permutation(9)[:3] for _ in range(20)])
    _, pos = od.positions(idx, 7)
    rows, w, dy = rng.normal(size=(60, 4)), rng.normal(size=(20, 3)), rng.normal(size=(20, 4))
    y, _ = od.combine_rows(rows, pos, w)
    drows, dw, _ = od.combine_backward(dy, rows, pos, w)
    total = (dy * y).sum()
    assert np.isclose((np.nan_to_num(drows) * rows).sum(), total) and np.isclose((dw * w).sum(), total)


def test_lora_by_hand():
    a = np.array([[[1.0, 0.0]], [[1.0, 1.0]]])            # two adapters of rank 1
    b = np.array([[[2.0], [0.0]], [[0.0], [3.0]]])
    x, base = np.array([[5.0, 7.0]] * 4), np.ones((4, 2))
    r = ol.lora(base, x, a, b, [1, 0, 2], [0, 1, 3, 3], [1.0, 0.5])
    assert np.array_equal(r["y"], [[1, 19], [11, 1], [11, 1], [np.nan, np.nan]], equal_nan=True)
    assert r["h"].ravel().tolist() == [6.0, 5.0, 5.0, 0.0]
    each = ol.lora(base, x, a, b, [1, 0, 0, -1], None, [1.0, 0.5])
    assert each["y"].tolist() == [[1, 19], [11, 1], [11, 1], [1, 1]]


def test_requests_of_bounds_out_of_order():
    assert ol.requests_of(6, [0, 4, 2, 9]).tolist() == [0, 0, 0, 0, 2, 2]
    assert ol.requests_of(5, [-3, 1, 1, 3]).tolist() == [0, 2, 2, -1, -1]
    assert ol.requests_of(3, None).tolist() == [0, 1, 2]


def test_drafts_by_hand():
    p = np.array([[[0.5, 0.25, 0.25], [0.0, 0.5, 0.5], [0.25, 0.75, 0.0]]])
    q = np.array([[[0.25, 0.5, 0.25], [0.5, 0.25, 0.25]]])

    def run(draft, ua, us, q=q, n=None):
        t, m = odr.verify(p, q, np.array([draft]), np.array([ua]), np.array([us]), n)
        return t[0].tolist(), int(m[0])

    assert run([0, 1], [0.9, 0.9], 0.3) == ([0, 1, 1], 2)          # both, then from p's last row
    assert run([1, 1], [0.49, 0.9], 0.2) == ([1, 1, 0], 2)
    assert run([1, 1], [0.5, 0.0], 0.9) == ([0, -1, -1], 0)        # r = (0.25, 0, 0)
    assert run([2, 0], [0.9, 0.0], 0.6) == ([2, 2, -1], 1)         # r = (0, 0.25, 0.25)
    assert run([0, 1], [0.9, 0.9], 0.3, n=[0]) == ([0, -1, -1], 0)
    assert run([1, 1], [0.24, 0.5], 0.99, q=None) == ([1, 2, -1], 1)   # looked up: u < p; 1 is out
    assert run([3, 1], [0.0, 0.0], 0.0) == ([0, -1, -1], 0)        # no token 3


def test_drafts_leave_the_targets_distribution():
    """All drafts, and random numbers at the middles of equal parts that the
    probabilities of this p and q are multiples of: counted, not sampled."""
    p, q = np.array([8, 2, 4, 2]) / 16, np.array([4, 4, 4, 4]) / 16
    share = np.zeros(4)
    mid = (np.arange(16) + 0.5) / 16
    for x, ua, us in itertools.product(range(4), mid, mid):
        t, _ = odr.verify(np.stack([p, p])[None], q[None, None], np.array([[x]]), np.array([[ua]]), np.array([us]))
        share[t[0, 0]] += q[x] / len(mid) ** 2
    assert np.allclose(share, p, atol=1e-12)
