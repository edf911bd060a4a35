"""GPU test of the rule for group bounds that are out of order: a bound below an
earlier one counts as that one, after each is clamped to the rows.  Against the
oracle with the running maximum of the bounds, the only result that is right.
Bars: those of test_gpu_mxfp4's products."""
import numpy as np
import pytest
import torch

import oracle.mxfp4 as mx
from parity import need_gpu
from test_gpu_mxfp4 import _bf, _close, _dev, _i32, _rand_mx

pytestmark = pytest.mark.gpu

CASES = [  # R, N, K, bounds
    (20, 32, 64, [-5, 6, 4, 12, 1 << 30]),               # the second group is empty, the third starts at 6
    (20, 32, 64, [9, 3, 3, 15, 15]),                     # rows before the first bound are in no group
    (40, 48, 96, [0, 40, 0, 20, 40]),                    # all rows in the first group
    (40, 48, 96, [0, 0, -1, -(1 << 31), 17]),            # one group, at the end
    (7, 16, 32, [(1 << 31) - 1, 0, 1, 2, 7]),            # no row in any group
]


@pytest.mark.parametrize("R,N,K,off", CASES)
def test_running_maximum(R, N, K, off):
    bf = _bf()
    dev = need_gpu()
    G = len(off) - 1
    rng = np.random.default_rng(R + N + K)
    ac, as_, av = _rand_mx(rng, R, K)
    wc, ws, wv = _rand_mx(rng, G, N, K)
    top = np.maximum.accumulate(np.clip(off, 0, R))
    ref, mag, cov = mx.product(av, wv, top)
    y = torch.full((R + 8, N), 7.0, device=dev)
    bf.mxfp4_linear(_dev(ac, as_), _dev(wc, ws), _i32(off), y=y[:R])
    ref[~cov], mag[~cov] = 7.0, 0.0
    _close(y[:R], ref, mag, K, torch.float32)
    assert (y[R:] == 7).all() and (y[:R][torch.from_numpy(~cov).to(dev)] == 7).all()
