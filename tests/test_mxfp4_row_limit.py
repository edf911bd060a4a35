"""Host checks (no GPU) of the most rows that a weight matrix of a 4-bit product
may have: the header states the limit, the library holds it, the binding names
it (a matrix of every token of a large vocabulary is past it)."""
import ctypes
import os
import re

import pytest
import torch

bf = pytest.importorskip("bit_expert_ffn_top_amd")
from bit_expert_ffn_top_amd._binding import Mxfp4C  # noqa: E402

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "bitffn_moe.h")
FAKE = 0x7F0000000000  # never dereferenced: no call below has a row to compute


def _limit():
    text = open(HEADER, encoding="utf-8").read()
    (value,) = re.findall(r"#define MOE_MAX_MX_OUT (\d+)", text)
    product = text[text.index("/* Products of 4-bit rows"):text.index("int moe_mxfp4_linear")]
    assert "MOE_MAX_MX_OUT" in product          # stated where the product is described
    return int(value)


@pytest.mark.parametrize("name", ["moe_mxfp4_linear", "moe_mxfp4_gate_up"])
def test_library_holds_the_header_limit(name):
    try:
        f = getattr(bf.lib(), name)
    except RuntimeError as e:
        pytest.skip(str(e))
    top = _limit()

    def call(rows):
        a, w = (ctypes.byref(Mxfp4C(1, n, 64, 0, FAKE, FAKE + 4096)) for n in (64, rows))
        return f(a, w, None, None, 1, 0, None, 0, None)

    assert call(top) == 0 and call(top + 64) == -1


@pytest.mark.parametrize("fn", [bf.mxfp4_linear, bf.mxfp4_gate_up])
def test_binding_names_the_limit(fn):
    top = _limit()
    assert str(top) in re.sub(r"[ ,\n]", "", fn.__doc__)

    def w(rows):
        return bf.Mxfp4(torch.empty((rows, 32), dtype=torch.uint8, device="meta"),
                        torch.empty((rows, 2), dtype=torch.uint8, device="meta"))

    with pytest.raises(ValueError, match=f"w: at most {top} rows expected, got {top + 64}"):
        fn(w(4), w(top + 64))
    with pytest.raises(ValueError, match="must be a device tensor"):
        fn(w(4), w(top))
