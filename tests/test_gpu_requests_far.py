"""GPU tests of the seams of indexes, counts and launches that only large calls of the
dispatch, the adapters and the verification of drafted tokens reach.
"""
import numpy as np
import pytest
import torch

import oracle.lora as ol
from parity import need_gpu
from test_gpu_lora import BF16, F32, _bf, _bound, _i32, _np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("one", [None, 0, 777_777, 65536 * 64 - 1])
@pytest.mark.parametrize("E", [5, 1024])
def test_dispatch_as_many_pairs_of_an_expert_as_a_part_holds(E, one):
    """65,536 tokens of 64 pairs, 32,768 in each part that is counted: all of the last
    expert, or all but one."""
    bf = _bf()
    dev = need_gpu()
    T, k = 65536, 64
    idx = torch.full((T * k,), E - 1, dtype=torch.int32, device=dev)
    want = torch.arange(T * k, dtype=torch.int32, device=dev)
    first = 0
    if one is not None:
        idx[one] = E - 2
        want[:one] += 1
        want[one] = 0
        first = 1
    x = torch.arange(T * 4, device=dev).view(T, 4).float()
    f = bf.dispatch(x, idx.view(T, k), E)
    assert torch.equal(f.pair_pos.view(-1), want)
    assert f.offsets.tolist() == [0] * (E - 1) + [first, T * k]
    rows = torch.empty_like(f.rows)
    rows[want.long()] = x.repeat_interleave(k, 0)
    assert torch.equal(f.rows, rows)


@pytest.mark.parametrize("S", [2, 70])
def test_adapters_more_tiles_than_a_grid_has_rows(S):
    """2.2 million rows, 68,750 tiles of 32: two requests, and seventy whose rows are
    gathered by adapter.  Rows on both sides of the seam, and both ends, have the bits
    that they have in a call of their own."""
    bf = _bf()
    dev = need_gpu()
    T, n = 2_200_000, 2
    g = torch.Generator(device=dev).manual_seed(S)
    x = torch.randn((T, 32), generator=g, device=dev).to(BF16)
    base = torch.randn((T, 16), generator=g, device=dev).to(BF16)
    a = torch.randn((n, 8, 32), generator=g, device=dev).to(BF16)
    b = torch.randn((n, 16, 8), generator=g, device=dev).to(BF16)
    bounds = np.concatenate([[0], 1000 + 13 * np.arange(S - 1), [T]])
    who = np.arange(S) % n
    y = bf.lora(base, x, a, b, _i32(who), seq_offsets=_i32(bounds))
    assert (T + 31) // 32 > 65536
    of = np.repeat(who, np.diff(bounds))
    seam = 65536 * 32
    for r0 in (0, 990, 1890, seam - 3000, seam - 40, seam + 40, T - 300):
        r1 = min(T, r0 + 400)
        alone = bf.lora(base[r0:r1].clone(), x[r0:r1].clone(), a, b, _i32(of[r0:r1]))
        assert torch.equal(y[r0:r1], alone), r0
    each = bf.lora(base[seam - 32768:seam + 32768].clone(), x[seam - 32768:seam + 32768].clone(), a, b,
                   _i32([int(of[seam])]), seq_offsets=_i32([0, 65536]))
    assert torch.equal(y[seam - 32768:seam + 32768], each)


def test_adapters_gathered_rows_far_apart():
    """Gathered rows whose byte offsets lie between 2^31 and 2^32."""
    bf = _bf()
    dev = need_gpu()
    T, d, n = 65000, 16384, 2
    assert 2 ** 31 < T * d * 4 < 2 ** 32
    g = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn((T, d), generator=g, device=dev)
    base = torch.randn((T, 16), generator=g, device=dev)
    a = (torch.randn((n, 8, d), generator=g, device=dev) / d ** 0.5).to(BF16)
    b = torch.randn((n, 16, 8), generator=g, device=dev).to(BF16)
    who = torch.randint(-1, n, (T,), generator=g, device=dev).int()
    y = bf.lora(base, x, a, b, who)
    some = [0, 1, 32766, 32767, 32768, 32769, 40001, T - 2, T - 1]
    r = ol.lora(_np(base[some]), _np(x[some]), _np(a), _np(b), who[some].cpu().numpy())
    assert (np.abs(_np(y[some]) - r["y"]) <= _bound(r, d, 8, F32)).all()
    for r0 in (0, 32700, T - 200):
        r1 = r0 + 200
        alone = bf.lora(base[r0:r1].clone(), x[r0:r1].clone(), a, b, who[r0:r1].clone())
        assert torch.equal(y[r0:r1], alone), r0


def test_drafts_of_more_requests_than_a_launch_takes():
    """32,770 requests with rows of more than 16,384 values: one value in each."""
    bf = _bf()
    dev = need_gpu()
    B, V = 32770, 16385
    p = torch.zeros((B, 1, V), device=dev)
    at = (torch.arange(B, device=dev) * 7919) % V
    p.view(B, V).scatter_(1, at[:, None], 0.25)
    p[32769] = 0.0
    none = torch.empty((B, 0), device=dev)
    tokens, accepted = bf.verify_drafts(p, None, none.int(), none, torch.full((B,), 0.5, device=dev))
    at[32769] = -1
    assert torch.equal(tokens[:, 0], at.int()) and not accepted.any()


def test_drafts_far_rows_of_p():
    """More than 2^32 values of p: the last request's row, and the first one's."""
    bf = _bf()
    dev = need_gpu()
    B, V = 257, 2 ** 24 - 1
    p = torch.zeros((B, 1, V), dtype=BF16, device=dev)
    assert (B - 1) * V > 2 ** 32 - 2 ** 24 and p.numel() > 2 ** 32
    p[0, 0, 3], p[-1, 0, 7], p[-1, 0, V - 1] = 1.0, 0.25, 0.75
    none = torch.empty((B, 0), device=dev)
    us = torch.full((B,), 0.5, device=dev)
    for u, last in ((0.5, V - 1), (0.125, 7)):
        us[-1] = u
        tokens, _ = bf.verify_drafts(p, None, none.int(), none, us)
        assert tokens[:, 0].tolist() == [3] + [-1] * (B - 2) + [last]


def test_drafts_far_rows_of_q():
    """More than 2^32 values of q and a draft that is refused: q's row decides."""
    bf = _bf()
    dev = need_gpu()
    B, V = 257, 2 ** 24 - 1
    p = torch.zeros((B, 2, V), dtype=BF16, device=dev)
    q = torch.zeros((B, 1, V), dtype=BF16, device=dev)
    assert q.numel() > 2 ** 32
    p[-1, 0, 5], p[-1, 0, V - 2] = 0.5, 0.5
    q[-1, 0, 5], q[-1, 0, V - 2] = 0.5, 0.25
    p[-1, 1, 11] = 1.0
    draft = torch.full((B, 1), 9, dtype=torch.int32, device=dev)
    ua, us = torch.full((B, 1), 0.5, device=dev), torch.full((B,), 0.125, device=dev)
    tokens, accepted = bf.verify_drafts(p, q, draft, ua, us)
    assert tokens[-1].tolist() == [V - 2, -1] and not accepted.any() and (tokens[:-1] == -1).all()
    draft[-1] = 5                                  # accepted: 0.5 * 0.5 < 0.5
    tokens, accepted = bf.verify_drafts(p, q, draft, ua, us)
    assert tokens[-1].tolist() == [5, 11] and accepted[-1].item() == 1
