"""GPU test of 4-bit products whose token codes are 2 GiB or more, so that the
kernel of full tiles, whose offsets into them have 32 bits, may not serve them.
Bars: those of test_gpu_mxfp4's products."""
import numpy as np
import pytest
import torch

import oracle.mxfp4 as mx
from parity import need_gpu
from test_gpu_mxfp4 import HALF_STEP, U, _bf, _dev, _i32, _np, _rand_mx, _silu_bound

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [262_143, 262_200])   # codes just below and just past 2^31 bytes
def test_rows_past_2_gib(rows):
    """66,000 rows gathered from all over A, its first and last ones among them;
    256 of the results against the oracle, both ends of A's among them."""
    bf = _bf()
    dev = need_gpu()
    K, N, R = 16384, 64, 66_000
    assert (rows * (K // 2) < 1 << 31) == (rows == 262_143)
    rng = np.random.default_rng(rows)
    g = torch.Generator(device=dev).manual_seed(rows)
    ac = torch.randint(0, 256, (rows, K // 2), generator=g, device=dev, dtype=torch.uint8)
    as_ = torch.randint(122, 127, (rows, K // 32), generator=g, device=dev, dtype=torch.uint8)
    wc, ws, wv = _rand_mx(rng, N, K, lo=118, hi=123)
    src = rng.integers(0, rows, R)
    src[:4], src[-4:] = [0, rows - 1, rows - 2, -1], [rows, rows - 1, 1, rows - 3]
    A, W, S = bf.Mxfp4(ac, as_), _dev(wc, ws), _i32(src)
    pick = np.unique(np.concatenate([np.arange(8), np.arange(R - 8, R), rng.integers(0, R, 240)]))
    at = torch.from_numpy(np.clip(src[pick], 0, rows - 1)).to(dev)
    av = mx.values(ac[at].cpu().numpy(), as_[at].cpu().numpy())
    av[(src[pick] < 0) | (src[pick] >= rows)] = 0.0
    ref, mag = av @ wv.T, np.abs(av) @ np.abs(wv.T)
    got = _np(bf.mxfp4_linear(A, W, row_src=S)[torch.from_numpy(pick).to(dev)])
    assert (np.abs(got - ref) <= 2 * K * U * mag * (1 + U) + U * np.abs(ref)).all()
    h = _np(bf.mxfp4_gate_up(A, W, row_src=S)[torch.from_numpy(pick).to(dev)])
    d = 2 * K * U * mag
    want = mx.silu(ref[:, 0::2]) * ref[:, 1::2]
    b = _silu_bound(ref[:, 0::2], ref[:, 1::2], d[:, 0::2], d[:, 1::2])
    assert (np.abs(h - want) <= b + HALF_STEP[torch.bfloat16] * (np.abs(want) + b) + 1e-40).all()
