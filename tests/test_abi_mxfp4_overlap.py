"""Host checks (no GPU): the 4-bit float, grouping and router-loss calls refuse a
buffer that they write and that is another of their buffers too; the workgroups
of a launch would read what others have written already."""
import ctypes
import itertools

import pytest
import torch

bf = pytest.importorskip("bit_expert_ffn_top_amd")
from bit_expert_ffn_top_amd._binding import Mxfp4C  # noqa: E402

BASE = 0x7F0000000000      # never dereferenced: every call below is refused by its host checks
EINVAL = -1


def _lib():
    try:
        return bf.lib()
    except RuntimeError as e:
        pytest.skip(str(e))


def _ptrs(names):
    """A far address of its own for each name."""
    return {n: BASE + (i << 40) for i, n in enumerate(names)}


def _mx(n, rows, cols, codes, scales):
    return ctypes.byref(Mxfp4C(n, rows, cols, 0, codes, scales))


def _quantize(p):
    return _lib().moe_mxfp4_quantize(p["x"], 1, 4, 64, p["codes"], p["scales"], None)


def _dequantize(p):
    return _lib().moe_mxfp4_dequantize(p["codes"], p["scales"], 4, 64, p["y"], 0, None)


def _product(name):
    def call(p):
        return getattr(_lib(), name)(_mx(1, 64, 64, p["ac"], p["as"]), _mx(2, 64, 64, p["wc"], p["ws"]), p["offsets"],
                                     p["row_src"], 1, 16, p["y"], 0, None)
    return call


def _decode(p):
    return _lib().moe_mxfp4_ffn_decode(_mx(8, 128, 96, p["gc"], p["gs"]), _mx(8, 96, 64, p["dc"], p["ds"]), -1, p["x"],
                                       2, 3, p["slot"], p["w"], p["y"], p["work"], 1 << 30, None)


def _group(p):
    return _lib().moe_group_pairs(p["idx"], 100, 2, 8, p["offsets"], p["pair_pos"], p["row_pair"], p["work"], 1 << 30,
                                  None)


def _balance(p):
    return _lib().moe_route_balance(p["logits"], p["idx"], 100, 8, 2, p["seq"], 3, p["mask"], p["balance"], p["z"],
                                    p["counts"], p["prob_sum"], p["n_tokens"], p["work"], 1 << 30, None)


CALLS = [  # call, what it writes, what it reads
    (_quantize, ["codes", "scales"], ["x"]),
    (_dequantize, ["y"], ["codes", "scales"]),
    (_product("moe_mxfp4_linear"), ["y"], ["ac", "as", "wc", "ws", "offsets", "row_src"]),
    (_product("moe_mxfp4_gate_up"), ["y"], ["ac", "as", "wc", "ws", "offsets", "row_src"]),
    (_decode, ["y", "work"], ["gc", "gs", "dc", "ds", "x", "slot", "w"]),
    (_group, ["offsets", "pair_pos", "row_pair", "work"], ["idx"]),
    (_balance, ["balance", "z", "counts", "prob_sum", "n_tokens", "work"], ["logits", "idx", "seq", "mask"]),
]
PAIRS = [(c, a, b) for c, written, read in CALLS
         for a, b in itertools.chain(itertools.combinations(written, 2), itertools.product(written, read))]
NAMES = {c: w + r for c, w, r in CALLS}


@pytest.mark.parametrize("call,a,b", PAIRS, ids=[f"{i}_{a}_{b}" for i, (_, a, b) in enumerate(PAIRS)])
def test_refused(call, a, b):
    if torch.cuda.is_available():
        pytest.skip("addresses of no memory: only where no launch could follow")
    p = _ptrs(NAMES[call])
    p[a] = p[b]
    assert call(p) == EINVAL
