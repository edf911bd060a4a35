"""GPU tests of combine_backward: the gradients that it allocates itself, where rows
that no pair uses have the gradient zero, whatever the memory held; and row lengths on
both sides of what a lane keeps of dy.
"""
import numpy as np
import pytest
import torch

import oracle.dispatch as od
from parity import need_gpu
from test_gpu_dispatch import BF16, F32, HALF_STEP, U, _bf, _dev, _np, _pos, _randn

pytestmark = pytest.mark.gpu


def _soil(n_bytes):
    """NaN in the memory that the next allocation of this size is likely to get."""
    for _ in range(4):
        torch.full((n_bytes // 4,), float("nan"), device=need_gpu())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,k,d,R,missing", [(1, 1, 4, 3, 0.0), (40, 6, 264, 240, 0.3), (700, 10, 72, 7000, 1.0),
                                             (5, 2, 16384, 64, 0.1), (0, 3, 64, 9, 0.0)])
@pytest.mark.parametrize("need_w", [True, False])
def test_rows_of_no_pair(T, k, d, R, missing, dtype, need_w):
    bf = _bf()
    pos = _pos(np.random.default_rng(T + d), T, k, R, missing)
    dy, rows, w = _randn(1, (T, d), dtype), _randn(2, (R, d), dtype), _randn(3, (T, k), F32)
    given = torch.zeros_like(rows)
    bf.combine_backward(dy, rows, _dev(pos), w, drows=given, need_w=False)
    _soil(rows.numel() * rows.element_size())
    drows, dw = bf.combine_backward(dy, rows, _dev(pos), w, need_w=need_w)
    assert torch.equal(drows, given) and (dw is None) != need_w
    none = np.setdiff1d(np.arange(R), pos.ravel())
    assert len(none) and not drows[torch.from_numpy(none).to(drows.device)].any()


def test_in_a_graph():
    """Cleared on every replay: another step's pairs leave nothing behind."""
    bf = _bf()
    rng = np.random.default_rng(3)
    pos = [_dev(_pos(rng, 30, 4, 120, 0.4)) for _ in range(3)]
    dy, rows, w = _randn(1, (30, 132), BF16), _randn(2, (120, 132), BF16), _randn(3, (30, 4), F32)
    want = [bf.combine_backward(dy, rows, p, w) for p in pos]
    live = pos[0].clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        drows, dw = bf.combine_backward(dy, rows, live, w)
    for i in (1, 2, 0, 2, 1):
        live.copy_(pos[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(drows, want[i][0]) and torch.equal(dw, want[i][1])
        assert torch.equal(bf.combine_backward(dy, rows, pos[i], w)[0], want[i][0])


@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("d", [252, 256, 260, 508, 512, 516, 1020, 1024, 1028, 2044, 2048, 2052, 2056, 4100])
def test_row_lengths(d, types):
    """Bars as in test_gpu_dispatch: one rounding of w dy to fp32 and one to the rows'
    type; d + 2 roundings of the terms of dw."""
    bf = _bf()
    gt, rt = types
    pos = _pos(np.random.default_rng(d), 9, 5, 60, 0.2)
    dy, rows, w = _randn(1, (9, d), gt), _randn(2, (60, d), rt), _randn(3, (9, 5), F32)
    drows, dw = bf.combine_backward(dy, rows, _dev(pos), w)
    ref, ref_w, mag = od.combine_backward(_np(dy), _np(rows), pos, _np(w))
    ref = np.nan_to_num(ref)
    assert (np.abs(_np(drows) - ref) <= (U + HALF_STEP[rt] * (1 + U)) * np.abs(ref)).all()
    assert (np.abs(_np(dw) - ref_w) <= (d + 2) * U * mag).all()


def test_on_a_given_stream():
    """The clearing runs on the stream that the call is given."""
    bf = _bf()
    pos = _dev(_pos(np.random.default_rng(5), 900, 8, 9000, 0.5))
    dy, rows, w = _randn(1, (900, 1024), BF16), _randn(2, (9000, 1024), BF16), _randn(3, (900, 8), F32)
    want = bf.combine_backward(dy, rows, pos, w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got = bf.combine_backward(dy, rows, pos, w, stream=side)
        side.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
