"""GPU tests of the router's balance and z losses, per-expert counts and logit
gradients against the fp64 oracle.

Bars, u = 2^-24.  A probability is exp(d) / sum, d = l - max: the difference
and its product with log2(e) round once each, which is a relative error of
2.2 |d| u of the exponential, and |d| <= 50 in these inputs wherever it is not 0
in fp32; the exponential and the division add a few u, the sum of E terms E u at
most: relative error at most P = (120 + E) u, or absolute 2^-125 where the
exponential underflows.
Sums over n rows add at most n u (relative to sums of positive terms).  lse
is max + log(sum): absolute error at most 4 u (|lse| + |max|) + (E + 4) u.
"""
import numpy as np
import pytest
import torch

import oracle.balance as ob
from parity import need_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 2.0 ** -125


def _bf():
    import bit_expert_ffn_top_amd as bf
    return bf


def _np(t):
    return None if t is None else t.detach().cpu().numpy().astype(np.float64)


def _case(T, E, k, seqs=None, masked=False, seed=0, scale=2.0):
    rng = np.random.default_rng(T * 1000 + E * 10 + k + seed)
    logits = (rng.normal(size=(T, E)) * scale).astype(np.float32)
    idx = np.argsort(-logits, 1, kind="stable")[:, :k].astype(np.int32)
    if seqs is not None:
        seqs = np.asarray(seqs, np.int32)
    mask = (rng.random(T) < 0.7).astype(np.uint8) if masked else None
    return logits, idx, seqs, mask


def _dev(*arrays):
    dev = need_gpu()
    return [None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev) for a in arrays]


def _check_forward(f, logits, idx, seqs, mask):
    E = logits.shape[1]
    ref = ob.route_balance(logits.astype(np.float64), idx, seqs, mask)
    assert np.array_equal(f.counts.cpu().numpy(), ref["counts"])
    assert np.array_equal(f.n_tokens.cpu().numpy(), ref["n_tokens"])
    n = ref["n_tokens"][:, None]
    rel = (120 + E + n) * U
    assert (np.abs(_np(f.prob_sum) - ref["prob_sum"]) <= rel * ref["prob_sum"] + n * TINY).all()
    assert (np.abs(_np(f.balance) - ref["balance"]) <= (rel[:, 0] + 8 * U) * ref["balance"] + TINY).all()
    big = np.abs(logits[np.isfinite(logits)]).max() if np.isfinite(logits).any() else 0.0
    dl = 8 * U * (big + 8) + (E + 4) * U                  # of one lse, |lse| <= |max| + log E
    zb = (2 * (big + 8) * dl + dl * dl) + (ref["n_tokens"] + 4) * U * ref["z"]
    assert (np.abs(_np(f.z) - ref["z"]) <= zb).all()
    return ref


SIZES = [  # T, E, k, sequence bounds, masked
    (1, 1, 1, None, False), (1, 512, 10, None, False), (4, 512, 10, [0, 1, 2, 4], False), (5, 3, 2, None, True),
    (64, 60, 6, [0, 10, 10, 64], True), (63, 61, 4, [3, 50, 60], False), (65, 64, 8, None, False),
    (131, 60, 6, [0, 20, 20, 77, 100, 131], True), (200, 100, 7, list(range(0, 201)), False),
    (257, 257, 3, [250, 257], True), (300, 1000, 64, [0, 299, 300], False), (1000, 1024, 64, [0, 0, 1000, 1000], True),
    (5000, 37, 5, [10, 2000, 2001, 4990], True), (9000, 512, 10, None, False), (4100, 128, 1, None, True),
    (40, 16, 2, [0, 1, 2, 3, 4, 5, 40], False),
]


@pytest.mark.parametrize("T,E,k,seqs,masked", SIZES, ids=[f"T{c[0]}_E{c[1]}_k{c[2]}_S{len(c[3] or [0, 0]) - 1}_m{int(c[4])}" for c in SIZES])
def test_forward_and_backward(T, E, k, seqs, masked):
    bf = _bf()
    logits, idx, seqs, mask = _case(T, E, k, seqs, masked)
    lg, ix, sq, mk = _dev(logits, idx, seqs, mask)
    f = bf.route_balance(lg, ix, sq, mk)
    again = bf.route_balance(lg, ix, sq, mk)
    for a, b in zip(f, again):
        assert torch.equal(a, b)
    ref = _check_forward(f, logits, idx, seqs, mask)
    S = len(ref["balance"])
    rng = np.random.default_rng(T + E)
    gb, gz = (rng.normal(size=S).astype(np.float32) for _ in range(2))
    e = np.exp(np.take_along_axis(logits, idx, 1).astype(np.float64))
    w = (e / e.sum(1, keepdims=True)).astype(np.float32)
    dw = rng.normal(size=(T, k)).astype(np.float32)
    dgb, dgz, dww, ddw = _dev(gb, gz, w, dw)
    for use in ("bzw", "b", "z", "w", ""):
        kw = dict(g_balance=dgb if "b" in use else None, g_z=dgz if "z" in use else None,
                  w=dww if "w" in use else None, dw=ddw if "w" in use else None)
        d = bf.route_backward(lg, ix, f.counts, f.n_tokens, seq_offsets=sq, mask=mk, **kw)
        _check_backward(d, logits, idx, ref["counts"], ref["n_tokens"], seqs, mask,
                        gb if "b" in use else None, gz if "z" in use else None,
                        w if "w" in use else None, dw if "w" in use else None)


def _check_backward(d, logits, idx, counts, n_tokens, seqs, mask, gb, gz, w, dw):
    """Each of the three terms may be off by its probability's relative error,
    the roundings of its sums and factors, taken on the magnitudes."""
    T, E = logits.shape
    k = idx.shape[1]
    f64 = [None if a is None else np.asarray(a, np.float64) for a in (gb, gz, w, dw)]
    ref = ob.route_backward(logits.astype(np.float64), idx, counts, n_tokens, *f64, seqs, mask)
    S = len(n_tokens)
    bound = np.full((T, E), 2.0 ** -120)
    rel = (130 + 2 * E) * U
    for s, rows in enumerate(ob.rows_of(T, seqs, S, mask)):
        n = max(int(n_tokens[s]), 1)
        for t in rows:
            p, lse = ob.softmax(logits[t].astype(np.float64))
            if gb is not None:
                c = np.abs(counts[s].astype(np.float64) - n * k // E)
                bound[t] += abs(float(gb[s])) * E / (k * n * n) * p * (c + (c * p).sum()) * 3 * rel
                # the oracle's own: c - sum c p in fp64, where it cancels (all
                # counts equal), keeps the roundings of p's and the sum's E
                # terms, 2^-53 each of at most the largest count
                bound[t] += abs(float(gb[s])) * E / (k * n * n) * p * 4 * E * 2.0 ** -53 * counts[s].max()
            if gz is not None and np.isfinite(lse):
                m = np.abs(logits[t][np.isfinite(logits[t])]).max()
                bound[t] += abs(float(gz[s])) * 2 / n * p * (3 * rel * abs(lse) + 8 * U * (m + abs(lse)) + rel)
            if w is not None:
                wt, dt = np.abs(w[t].astype(np.float64)), np.abs(dw[t].astype(np.float64))
                v = wt * (dt + (wt * dt).sum()) * (k + 8) * U
                for i in range(k):
                    if 0 <= idx[t, i] < E:
                        bound[t, idx[t, i]] += 2 * v[i]
    bound += 4 * U * np.abs(ref)
    err = np.abs(_np(d) - ref)
    assert (err <= bound).all(), float((err / bound).max())


def test_backward_against_differences():
    """The gradient against central differences of the oracle's losses: error
    of the differences h^2 max|f'''| / 6 + 1e-16 |f| / h < 1e-8, of the kernel
    far less than the 1e-5 relative bar."""
    bf = _bf()
    logits, idx, seqs, mask = _case(11, 13, 3, [1, 5, 5, 10], True, scale=1.0)
    rng = np.random.default_rng(0)
    gb, gz, dw = (rng.normal(size=s).astype(np.float32) for s in (3, 3, (11, 3)))
    base = logits.astype(np.float64)
    part = np.zeros(11, bool)
    for rows in ob.rows_of(11, seqs, 3, mask):
        part[rows] = True

    def weights(l):
        e = np.exp(np.take_along_axis(l, idx, 1))
        return e / e.sum(1, keepdims=True)

    def total(l):
        g = ob.route_balance(l, idx, seqs, mask)
        return (gb * g["balance"]).sum() + (gz * g["z"]).sum() + (weights(l) * dw)[part].sum()

    lg, ix, sq, mk, dgb, dgz, ddw, ww = _dev(logits, idx, seqs, mask, gb, gz, dw, weights(base).astype(np.float32))
    f = bf.route_balance(lg, ix, sq, mk)
    d = _np(bf.route_backward(lg, ix, f.counts, f.n_tokens, dgb, dgz, ww, ddw, sq, mk))
    h = 1e-6
    for t in range(11):
        for e in range(13):
            up, dn = base.copy(), base.copy()
            up[t, e] += h
            dn[t, e] -= h
            num = (total(up) - total(dn)) / (2 * h)
            assert abs(num - d[t, e]) <= 1e-5 * max(abs(num), 0.1), (t, e)


@pytest.mark.parametrize("E", [6, 64, 300, 512])
def test_masked_rows_hold_anything(E):
    """NaN and infinities in rows that take no part (masked, before the first
    and behind the last sequence) change nothing and get a gradient of 0."""
    bf = _bf()
    T, k = 70, 3
    logits, idx, seqs, mask = _case(T, E, k, [5, 30, 60], True)
    part = np.zeros(T, bool)
    for rows in ob.rows_of(T, seqs, 2, mask):
        part[rows] = True
    bad = logits.copy()
    bad[~part] = np.array([np.nan, np.inf, -np.inf])[np.arange((~part).sum()) % 3][:, None]
    bad_idx = idx.copy()
    bad_idx[~part] = 1 << 30
    w = np.full((T, k), 1 / k, np.float32)
    dw = np.random.default_rng(1).normal(size=(T, k)).astype(np.float32)
    w[~part], dw[~part] = np.nan, np.inf
    lg, ix, bl, bi, sq, mk, ww, dd = _dev(logits, idx, bad, bad_idx, seqs, mask, w, dw)
    f, g = bf.route_balance(lg, ix, sq, mk), bf.route_balance(bl, bi, sq, mk)
    for a, b in zip(f, g):
        assert torch.equal(a, b)
    ones = torch.ones(2, device=lg.device)
    d = bf.route_backward(bl, bi, g.counts, g.n_tokens, ones, ones, ww, dd, sq, mk)
    assert not d[torch.from_numpy(~part).to(d.device)].any()
    assert torch.isfinite(d).all() and d[torch.from_numpy(part).to(d.device)].any()
    # the same with a bool mask
    for a, b in zip(f, bf.route_balance(bl, bi, sq, mk.bool())):
        assert torch.equal(a, b)


def test_infinite_and_nan_logits():
    """Masked experts (-inf, the type's lowest value), rows of nothing but
    -inf, +inf, NaN: the conventions of the header, against the oracle."""
    bf = _bf()
    T, E, k = 9, 12, 2
    logits, idx, _, _ = _case(T, E, k)
    logits[0, 3:] = -np.inf
    logits[1, :] = -np.inf
    logits[2, 4] = np.inf
    logits[3, 4:6] = np.inf
    logits[4, 2] = np.nan
    logits[5, :] = np.nan
    logits[6, 5:] = np.finfo(np.float32).min
    logits[7, :] = np.finfo(np.float32).min
    lg, ix = _dev(logits, idx)
    f = bf.route_balance(lg, ix)
    ref = ob.route_balance(logits.astype(np.float64), idx)
    assert np.array_equal(f.counts.cpu().numpy(), ref["counts"])
    assert np.abs(_np(f.prob_sum) - ref["prob_sum"]).max() <= 200 * U * T
    # the row at the lowest value has a finite lse of -3.4e38, whose square
    # passes fp32's range: z is infinite
    assert np.isinf(_np(f.z)).all()
    keep = [0, 1, 2, 3, 4, 5, 6, 8]
    lg, ix = _dev(logits[keep], idx[keep])
    f = bf.route_balance(lg, ix)
    ref = ob.route_balance(logits[keep].astype(np.float64), idx[keep])
    assert np.abs(_np(f.z) - ref["z"]).max() <= 400 * U * ref["z"].max()
    one = torch.ones(1, device=lg.device)
    d = _np(bf.route_backward(lg, ix, f.counts, f.n_tokens, one, one))
    want = ob.route_backward(logits[keep].astype(np.float64), idx[keep], ref["counts"], ref["n_tokens"], [1.0], [1.0])
    assert np.isfinite(d).all()
    assert np.abs(d - want).max() <= 1000 * U * np.abs(want).max()


def test_ids_outside_and_repeated():
    bf = _bf()
    T, E, k = 20, 7, 6
    logits, idx, _, _ = _case(T, E, k)
    idx[0] = [2, 2, 2, 2, 2, 2]
    idx[1] = [-1, 7, 1 << 30, 0, 0, -(1 << 31)]
    idx[2] = [6, 1, 6, 1, 6, 3]
    lg, ix = _dev(logits, idx)
    f = bf.route_balance(lg, ix)
    ref = _check_forward(f, logits, idx, None, None)
    rng = np.random.default_rng(3)
    w, dw = rng.random((T, k)).astype(np.float32), rng.normal(size=(T, k)).astype(np.float32)
    ww, dd = _dev(w, dw)
    one = torch.ones(1, device=lg.device)
    a = bf.route_backward(lg, ix, f.counts, f.n_tokens, one, one, ww, dd)
    for _ in range(3):
        assert torch.equal(a, bf.route_backward(lg, ix, f.counts, f.n_tokens, one, one, ww, dd))
    _check_backward(a, logits, idx, ref["counts"], ref["n_tokens"], None, None, np.ones(1, np.float32),
                    np.ones(1, np.float32), w, dw)


def test_nothing_takes_part():
    bf = _bf()
    dev = need_gpu()
    logits, idx, _, _ = _case(80, 20, 3)
    lg, ix, sq = _dev(logits, idx, np.zeros(7, np.int32))
    for f in (bf.route_balance(lg, ix, sq), bf.route_balance(lg, ix, mask=torch.zeros(80, dtype=torch.uint8, device=dev)),
              bf.route_balance(lg[:0], ix[:0]), bf.route_balance(lg[:0], ix[:0], sq),
              bf.route_balance(lg[:9].contiguous(), ix[:9].contiguous(), sq[:3].contiguous())):
        for t in f:
            assert not t.any()
    f = bf.route_balance(lg, ix, sq)
    one = torch.ones(6, device=dev)
    d = torch.full((80, 20), 7.0, device=dev)
    bf.route_backward(lg, ix, f.counts, f.n_tokens, one, one, seq_offsets=sq, dlogits=d)
    assert not d.any()
    assert bf.route_backward(lg[:0], ix[:0], f.counts[:1].contiguous(), f.n_tokens[:1].contiguous(),
                             one[:1].clone()).shape == (0, 20)


def test_counts_summed_over_processes():
    """Counts and row counts that another process's rows joined: the gradient
    of the loss over both batches, of this batch's rows."""
    bf = _bf()
    logits, idx, _, _ = _case(50, 16, 4)
    other, oidx, _, _ = _case(70, 16, 4, seed=5)
    lg, ix, l2, i2 = _dev(logits, idx, other, oidx)
    a, b = bf.route_balance(lg, ix), bf.route_balance(l2, i2)
    one = torch.ones(1, device=lg.device)
    d = bf.route_backward(lg, ix, a.counts + b.counts, a.n_tokens + b.n_tokens, one)
    both = bf.route_balance(torch.cat([lg, l2]), torch.cat([ix, i2]))
    e = bf.route_backward(torch.cat([lg, l2]), torch.cat([ix, i2]), both.counts, both.n_tokens, one)
    assert torch.equal(d, e[:50])


def test_router_training_step():
    """route_topk -> route_balance -> route_backward as a step uses them, on a
    side stream and in a replayed graph, with the eager bits."""
    bf = _bf()
    dev = need_gpu()
    T, E, k = 300, 60, 6
    logits, _, seqs, mask = _case(T, E, k, [0, 100, 180, 300], True)
    lg, sq, mk = _dev(logits, seqs, mask)
    dw = torch.randn((T, k), generator=torch.Generator().manual_seed(1)).to(dev)
    gb, gz = torch.full((3,), 0.01, device=dev), torch.full((3,), 0.001, device=dev)

    def step(lg, stream=None):
        idx, w = bf.route_topk(lg, k, stream=stream)
        f = bf.route_balance(lg, idx, sq, mk, stream=stream)
        d = bf.route_backward(lg, idx, f.counts, f.n_tokens, gb, gz, w, dw, sq, mk, stream=stream)
        return (*f, d)

    ins = [lg, -lg, lg.flip(0).contiguous()]
    eager = [step(x) for x in ins]
    idx, w = (t.cpu().numpy() for t in bf.route_topk(lg, k))
    ref = _check_forward(bf.RouteBalance(*eager[0][:5]), logits, idx, seqs, mask)
    _check_backward(eager[0][5], logits, idx, ref["counts"], ref["n_tokens"], seqs, mask, _np(gb).astype(np.float32),
                    _np(gz).astype(np.float32), w, dw.cpu().numpy())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        out = step(lg)
    f = bf.route_balance(lg, torch.from_numpy(idx).to(dev), sq, mk)
    torch.cuda.synchronize()
    idx_d = torch.from_numpy(idx).to(dev)
    torch.cuda.synchronize()
    g = bf.route_balance(lg, idx_d, sq, mk, stream=side)
    torch.cuda.synchronize()
    for a, b, c, e in zip(out[:5], f, g, eager[0][:5]):
        assert torch.equal(a, e) and torch.equal(b, e) and torch.equal(c, e)
    assert torch.equal(out[5], eager[0][5])
    static = lg.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(static)
    for i in (1, 2, 0, 0, 2):
        static.copy_(ins[i])
        graph.replay()
        torch.cuda.synchronize()
        now = step(ins[i])
        for a, b, c in zip(got, eager[i], now):
            assert torch.equal(a, b) and torch.equal(c, b), i


def test_more_than_2_31_logits():
    """Row offsets past 2^31 elements."""
    bf = _bf()
    dev = need_gpu()
    T, E = 2_100_000, 1024
    lg = torch.zeros((T, E), device=dev)
    ix = torch.zeros((T, 1), dtype=torch.int32, device=dev)
    lg[-1, 5] = 20.0
    ix[-1] = 5
    sq = torch.tensor([T - 2, T - 1, T], dtype=torch.int32, device=dev)
    f = bf.route_balance(lg, ix, sq)
    assert f.counts[0, 0] == 1 and f.counts[1, 5] == 1 and int(f.counts.sum()) == 2
    assert abs(float(f.prob_sum[1, 5]) - 1.0) < 1e-5 and abs(float(f.prob_sum[0, 9]) * E - 1) < 1e-4
    one = torch.ones(2, device=dev)
    d = bf.route_backward(lg, ix, f.counts, f.n_tokens, None, one, seq_offsets=sq)
    assert not d[:T - 2].any()
    assert abs(float(d[-1, 5]) - 2 * 20.0) < 1e-2 and abs(float(d[-2, 3]) * E - 2 * np.log(E)) < 1e-3


def test_device_refusals():
    bf = _bf()
    dev = need_gpu()
    lg, ix = torch.zeros((4, 8), device=dev), torch.zeros((4, 2), dtype=torch.int32, device=dev)
    with pytest.raises(ValueError, match="contiguous"):
        bf.route_balance(lg.t().contiguous().t(), ix)
    with pytest.raises(ValueError, match="idx must be"):
        bf.route_balance(lg, ix.long())
    with pytest.raises(ValueError, match="must be a device tensor"):
        bf.route_balance(lg, ix, mask=torch.zeros(4, dtype=torch.uint8))
    with pytest.raises(bf.MoeError, match="workspace"):
        bf.route_balance(torch.zeros((100, 8), device=dev), torch.zeros((100, 2), dtype=torch.int32, device=dev),
                         ws=torch.empty((16,), dtype=torch.uint8, device=dev))
    with pytest.raises(bf.MoeError, match="invalid argument"):
        bf.route_backward(lg, ix, g_balance=torch.ones(1, device=dev))
