"""Pins of the balance-loss oracle: closed forms, and the gradient against
differences of the losses."""
import numpy as np

import oracle.balance as ob


def test_even_router_has_loss_one():
    T, E, k = 12, 6, 2
    logits = np.zeros((T, E))
    idx = np.array([[(k * t + i) % E for i in range(k)] for t in range(T)])
    f = ob.route_balance(logits, idx)
    assert np.allclose(f["balance"], 1.0) and np.allclose(f["z"], np.log(E) ** 2)
    assert f["counts"].tolist() == [[T * k // E] * E] and np.allclose(f["prob_sum"], T / E)


def test_collapsed_router_has_loss_E_over_k():
    logits = np.full((5, 4), -np.inf)
    logits[:, 2] = 3.0
    f = ob.route_balance(logits, np.full((5, 1), 2))
    assert np.allclose(f["balance"], 4.0) and np.allclose(f["z"], 9.0)


def test_rows_that_leave_nothing():
    logits = np.array([[np.nan, -np.inf], [np.inf, np.inf], [0.0, 0.0]])
    f = ob.route_balance(logits, np.array([[0], [1], [5]]))
    assert np.allclose(f["prob_sum"], [[1.5, 1.5]]) and np.allclose(f["z"], np.log(2) ** 2 / 3)
    assert f["counts"].tolist() == [[1, 1]]


def test_gradient_against_differences():
    rng = np.random.default_rng(1)
    T, E, k, off = 9, 7, 3, [1, 4, 4, 8]
    mask = np.array([1, 1, 0, 1, 1, 1, 1, 0, 1])
    logits = rng.normal(size=(T, E))
    idx = np.argsort(-logits, 1)[:, :k]
    gb, gz, dw = rng.normal(size=3), rng.normal(size=3), rng.normal(size=(T, k))
    f = ob.route_balance(logits, idx, off, mask)
    part = np.zeros(T, bool)
    for rows in ob.rows_of(T, off, 3, mask):
        part[rows] = True

    def weights(l):
        e = np.exp(np.take_along_axis(l, idx, 1))
        return e / e.sum(1, keepdims=True)

    def total(l):
        g = ob.route_balance(l, idx, off, mask)
        return (gb * g["balance"]).sum() + (gz * g["z"]).sum() + (weights(l) * dw)[part].sum()

    d = ob.route_backward(logits, idx, f["counts"], f["n_tokens"], gb, gz, weights(logits), dw, off, mask)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            up, dn = logits.copy(), logits.copy()
            up[t, e] += h
            dn[t, e] -= h
            # central differences in fp64: truncation h^2, rounding 1e-16 / h
            assert abs((total(up) - total(dn)) / (2 * h) - d[t, e]) < 1e-8
