"""GPU test of the 4-bit decode FFN with more experts than one round of the down
product's wavefronts, twice over: 16 wavefronts take an expert each, ask for their
next one's rows before they use them, and come back to the first set of registers
with the 33rd expert.  Bars: those of test_gpu_mxfp4's decode cases."""
import numpy as np
import pytest
import torch

from parity import need_gpu
from test_gpu_mxfp4 import _bf, _check_decode, _decode_case, _dev, _i32

pytestmark = pytest.mark.gpu

CASES = [  # T, k, n, d, F, shared: rows of up to 16, 32 and 64 blocks of F
    (1, 64, 70, 64, 96, False), (1, 64, 70, 64, 96, True), (4, 16, 64, 96, 96, True), (4, 16, 64, 128, 96, False),
    (1, 64, 64, 64, 544, True), (4, 16, 64, 64, 1056, True), (2, 32, 66, 2048, 768, True), (3, 21, 63, 4096, 2048, False),
]


@pytest.mark.parametrize("case", CASES, ids=["T%d_k%d_n%d_d%d_F%d_s%d" % c for c in CASES])
def test_more_than_32_experts(case):
    bf = _bf()
    dev = need_gpu()
    (gc, gs, gv), (dc, ds, dv), x, slot, w, shared = _decode_case(*case)
    assert len(np.unique(slot)) + (shared >= 0) > 32
    args = (_dev(gc, gs), _dev(dc, ds), torch.from_numpy(x).to(dev), _i32(slot).reshape(slot.shape),
            torch.from_numpy(w).to(dev))
    y = bf.mxfp4_ffn_decode(*args, shared_slot=shared)
    assert torch.equal(y, bf.mxfp4_ffn_decode(*args, shared_slot=shared))
    _check_decode(y, gv, dv, x, slot, w, shared)
    for t in range(x.shape[0]):         # and each token with the bits it has alone
        one = bf.mxfp4_ffn_decode(args[0], args[1], *(a[t:t + 1].clone() for a in args[2:]), shared_slot=shared)
        assert torch.equal(y[t], one[0]), t
