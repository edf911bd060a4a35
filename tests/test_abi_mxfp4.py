"""Host checks (no GPU) of the 4-bit float products, the grouping and the
router's losses: the C entry points refuse bad arguments before any HIP call,
the binding refuses wrong shapes, types and places before the library."""
import ctypes

import pytest
import torch

bf = pytest.importorskip("bit_expert_ffn_top_amd")
from bit_expert_ffn_top_amd._binding import Mxfp4C  # noqa: E402

FAKE = 0x7F0000000000  # never dereferenced: every call below fails its host checks
EINVAL, EALIGN, ENOSPC = -1, -2, -4


def _lib():
    try:
        return bf.lib()
    except RuntimeError as e:
        pytest.skip(str(e))


def _p(off=0):
    return ctypes.c_void_p(FAKE + off)


S0 = ctypes.c_void_p(0)


def _mx(n=1, rows=64, cols=64, reserved=0, codes=FAKE, scales=FAKE + 4096):
    return ctypes.byref(Mxfp4C(n, rows, cols, reserved, codes, scales))


def test_quantize_refusals():
    f = _lib().moe_mxfp4_quantize
    assert f(_p(), 2, 4, 64, _p(), _p(), S0) == EINVAL          # unknown type
    assert f(_p(), 0, -1, 64, _p(), _p(), S0) == EINVAL
    assert f(_p(), 0, 1 << 24, 64, _p(), _p(), S0) == EINVAL
    for cols in (0, 16, 33, 16384 + 32, -32):
        assert f(_p(), 0, 4, cols, _p(), _p(), S0) == EINVAL, cols
    assert f(None, 0, 4, 64, _p(), _p(), S0) == EINVAL
    assert f(_p(), 0, 4, 64, None, _p(), S0) == EINVAL
    assert f(_p(), 0, 4, 64, _p(), None, S0) == EINVAL
    assert f(_p(4), 0, 4, 64, _p(), _p(), S0) == EALIGN
    assert f(_p(), 0, 4, 64, _p(8), _p(), S0) == EALIGN
    assert f(_p(), 0, 4, 64, _p(), _p(1), S0) == EALIGN
    assert f(None, 0, 0, 64, None, None, S0) == 0               # no rows: nothing to do


def test_dequantize_refusals():
    f = _lib().moe_mxfp4_dequantize
    assert f(_p(), _p(), 4, 64, _p(), 3, S0) == EINVAL
    assert f(_p(), _p(), 4, 48, _p(), 0, S0) == EINVAL
    assert f(_p(), _p(), 4, 64, None, 0, S0) == EINVAL
    assert f(_p(), _p(), 4, 64, _p(2), 1, S0) == EALIGN
    assert f(None, None, 0, 64, None, 0, S0) == 0


@pytest.mark.parametrize("gated", [False, True])
def test_product_refusals(gated):
    f = _lib().moe_mxfp4_gate_up if gated else _lib().moe_mxfp4_linear

    def call(A=None, W=None, offsets=None, row_src=None, div=1, R=16, y=_p(8192), dt=0):
        return f(A or _mx(), W or _mx(), offsets, row_src, div, R, y, dt, S0)

    assert f(None, _mx(), None, None, 1, 16, _p(), 0, S0) == EINVAL
    assert f(_mx(), None, None, None, 1, 16, _p(), 0, S0) == EINVAL
    assert call(A=_mx(n=2)) == EINVAL                       # A is one matrix
    assert call(A=_mx(cols=96)) == EINVAL                   # columns differ
    assert call(W=_mx(rows=40 if not gated else 48)) == EINVAL
    assert call(W=_mx(rows=65536 + 64)) == EINVAL
    assert call(W=_mx(n=2)) == EINVAL                       # groups without bounds
    assert call(W=_mx(n=1025), offsets=_p()) == EINVAL
    assert call(W=_mx(reserved=1)) == EINVAL
    assert call(A=_mx(rows=0)) == EINVAL
    assert call(A=_mx(codes=None)) == EINVAL
    assert call(A=_mx(codes=FAKE + 4)) == EALIGN
    assert call(W=_mx(scales=FAKE + 1)) == EALIGN
    assert call(R=-1) == EINVAL and call(R=1 << 24) == EINVAL
    assert call(R=65) == EINVAL                             # more rows than A without row_src
    assert call(div=0, row_src=_p()) == EINVAL
    assert call(dt=2) == EINVAL
    assert call(y=None) == EINVAL and call(y=_p()) == EINVAL    # aliases A's codes
    assert call(y=_p(8)) == EALIGN
    assert call(offsets=_p(4)) == EALIGN and call(row_src=_p(4)) == EALIGN
    assert call(R=0, y=None) == 0


def test_decode_refusals():
    lib = _lib()
    need = lib.moe_mxfp4_ffn_decode_workspace_bytes(4, 10, 64)
    assert need >= 4 * 11 * 64 * 4
    for bad in ((0, 10, 64), (5, 10, 64), (4, 17, 64), (1, 65, 64), (1, -1, 64), (1, 10, 48), (1, 10, 4128)):
        assert lib.moe_mxfp4_ffn_decode_workspace_bytes(*bad) == 0, bad

    def call(GU=None, D=None, shared=-1, x=_p(), T=4, k=10, slot=_p(), w=_p(), y=_p(8192),
             ws=_p(), nb=need):
        return lib.moe_mxfp4_ffn_decode(GU or _mx(8, 128, 96), D or _mx(8, 96, 64), shared, x, T, k,
                                        slot, w, y, ws, nb, S0)

    assert call(GU=_mx(7, 128, 96)) == EINVAL
    assert call(GU=_mx(8, 64, 96)) == EINVAL
    assert call(D=_mx(8, 64, 64)) == EINVAL
    assert call(GU=_mx(8, 128, 4128), D=_mx(8, 4128, 64)) == EINVAL
    assert call(shared=8) == EINVAL and call(shared=-2) == EINVAL
    assert call(T=0) == EINVAL and call(T=5) == EINVAL and call(T=4, k=17) == EINVAL
    assert call(x=None) == EINVAL and call(y=None) == EINVAL and call(ws=None) == EINVAL
    assert call(slot=None) == EINVAL and call(w=None) == EINVAL
    assert call(y=_p()) == EINVAL                           # y aliases x
    assert call(x=_p(4)) == EALIGN and call(ws=_p(16)) == EALIGN and call(slot=_p(8)) == EALIGN
    assert call(nb=need - 1) == ENOSPC


def test_group_refusals():
    lib = _lib()
    need = lib.moe_group_workspace_bytes(100, 8)
    assert need > 0 and lib.moe_group_workspace_bytes(0, 8) == 0
    assert lib.moe_group_workspace_bytes(65537, 8) == 0 and lib.moe_group_workspace_bytes(4, 1025) == 0

    def call(idx=_p(), T=100, k=2, E=8, off=_p(), pos=_p(), rows=_p(), ws=_p(), nb=need):
        return lib.moe_group_pairs(idx, T, k, E, off, pos, rows, ws, nb, S0)

    assert call(T=0) == EINVAL and call(T=65537) == EINVAL
    assert call(k=0) == EINVAL and call(k=65) == EINVAL
    assert call(E=0) == EINVAL and call(E=1025) == EINVAL
    assert call(idx=None) == EINVAL and call(off=None) == EINVAL and call(rows=None) == EINVAL
    assert call(ws=None) == EINVAL and call(ws=_p(16)) == EALIGN and call(pos=_p(4)) == EALIGN
    assert call(nb=need - 1) == ENOSPC


def test_balance_refusals():
    lib = _lib()
    need = lib.moe_route_balance_workspace_bytes(100, 8, 3)
    assert need > 0
    for bad in ((-1, 8, 1), (1 << 24, 8, 1), (4, 0, 1), (4, 1025, 1), (4, 8, 0), (4, 8, 65537)):
        assert lib.moe_route_balance_workspace_bytes(*bad) == 0, bad

    def call(lg=_p(), idx=_p(), T=100, E=8, k=2, seq=_p(), S=3, mask=None, b=_p(), z=_p(), c=_p(),
             p=_p(), n=_p(), ws=_p(), nb=need):
        return lib.moe_route_balance(lg, idx, T, E, k, seq, S, mask, b, z, c, p, n, ws, nb, S0)

    assert call(lg=None) == EINVAL and call(idx=None) == EINVAL
    assert call(T=-1) == EINVAL and call(T=1 << 24) == EINVAL
    assert call(E=0) == EINVAL and call(E=1025) == EINVAL
    assert call(k=0) == EINVAL and call(k=65) == EINVAL
    assert call(seq=None) == EINVAL                       # three sequences without bounds
    assert call(S=0) == EINVAL and call(S=65537) == EINVAL
    for name in "bzcpn":
        assert call(**{name: None}) == EINVAL and call(**{name: _p(8)}) == EALIGN, name
    assert call(mask=_p(1)) == EALIGN and call(seq=_p(4)) == EALIGN and call(lg=_p(4)) == EALIGN
    assert call(ws=None) == EINVAL and call(ws=_p(128)) == EALIGN and call(nb=need - 1) == ENOSPC


def test_backward_refusals():
    lib = _lib()

    def call(lg=_p(), idx=_p(), T=100, E=8, k=2, seq=_p(), S=3, mask=None, c=_p(), n=_p(), gb=_p(),
             gz=_p(), w=_p(), dw=_p(), d=_p(65536)):
        return lib.moe_route_backward(lg, idx, T, E, k, seq, S, mask, c, n, gb, gz, w, dw, d, S0)

    assert call(w=None) == EINVAL and call(dw=None) == EINVAL      # one without the other
    assert call(c=None) == EINVAL and call(n=None) == EINVAL
    assert call(gb=None, c=None, n=None) == EINVAL                 # z needs the row counts
    assert call(d=None) == EINVAL and call(d=_p()) == EINVAL       # aliases the logits
    assert call(d=_p(65536 + 4)) == EALIGN and call(dw=_p(8)) == EALIGN
    assert call(k=65) == EINVAL and call(E=1025) == EINVAL and call(S=0) == EINVAL
    assert call(T=0, lg=None, idx=None, d=None) == 0


# --- the binding ----------------------------------------------------------------


def _raises(match, fn, *a, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


def _q(*shape):
    return bf.Mxfp4(torch.zeros(shape[:-1] + (shape[-1] // 2,), dtype=torch.uint8),
                    torch.zeros(shape[:-1] + (shape[-1] // 32,), dtype=torch.uint8))


def test_binding_quantize():
    _raises("2 or 3 dimensions", bf.mxfp4_quantize, torch.zeros(32))
    _raises("multiple of 32", bf.mxfp4_quantize, torch.zeros(2, 48))
    _raises("float32 or bfloat16", bf.mxfp4_quantize, torch.zeros((2, 32), dtype=torch.float16))
    _raises("out.scales: shape", bf.mxfp4_quantize, torch.zeros(2, 64),
            bf.Mxfp4(torch.zeros((2, 32), dtype=torch.uint8), torch.zeros((2, 3), dtype=torch.uint8)))
    _raises("x must be a device tensor", bf.mxfp4_quantize, torch.zeros(2, 64))
    _raises("q.scales: shape", bf.mxfp4_dequantize,
            bf.Mxfp4(torch.zeros((2, 32), dtype=torch.uint8), torch.zeros((2, 1), dtype=torch.uint8)))
    _raises("float32 or bfloat16", bf.mxfp4_dequantize, _q(2, 64), torch.float16)
    _raises("q.codes must be a device tensor", bf.mxfp4_dequantize, _q(2, 64))


def test_binding_products():
    i32 = dict(dtype=torch.int32)
    for fn in (bf.mxfp4_linear, bf.mxfp4_gate_up):
        _raises("one matrix", fn, _q(2, 4, 64), _q(1, 64, 64))
        _raises("64 columns, w 96", fn, _q(4, 64), _q(1, 64, 96))
        _raises("offsets are needed", fn, _q(4, 64), _q(2, 64, 64))
        _raises(r"offsets: shape \(3,\)", fn, _q(4, 64), _q(2, 64, 64), torch.zeros(2, **i32))
        _raises("row_src: shape", fn, _q(4, 64), _q(64, 64), None, torch.zeros((2, 2), **i32))
        _raises("y must be float32 or bfloat16", fn, _q(4, 64), _q(64, 64), dtype=torch.float16)
        _raises("a.codes must be a device tensor", fn, _q(4, 64), _q(64, 64))
    _raises(r"y: shape \(4, 64\)", bf.mxfp4_linear, _q(4, 64), _q(64, 64), y=torch.zeros(4, 32))


def test_binding_decode():
    x, sl, w = torch.zeros(2, 64), torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, 3)
    _raises("down: ", bf.mxfp4_ffn_decode, _q(4, 64, 64), _q(4, 64, 64), x, sl, w)
    _raises("x: shape", bf.mxfp4_ffn_decode, _q(4, 64, 64), _q(4, 64, 32), torch.zeros(2, 32), sl, w)
    _raises("slot: shape", bf.mxfp4_ffn_decode, _q(4, 64, 64), _q(4, 64, 32), x, sl[:1], w)
    _raises("w: shape", bf.mxfp4_ffn_decode, _q(4, 64, 64), _q(4, 64, 32), x, sl, w[:, :2])
    _raises("x must be a device", bf.mxfp4_ffn_decode, _q(4, 64, 64), _q(4, 64, 32), x, sl, w)


def test_binding_balance():
    lg, idx = torch.zeros(4, 8), torch.zeros((4, 2), dtype=torch.int32)
    for fn in (bf.route_balance, bf.route_backward):
        _raises("logits: shape", fn, torch.zeros(8), idx)
        _raises("idx: shape", fn, lg, idx[:3])
        _raises("seq_offsets: at least 2", fn, lg, idx, seq_offsets=torch.zeros(1, dtype=torch.int32))
        _raises("mask: shape", fn, lg, idx, mask=torch.zeros(3, dtype=torch.uint8))
        _raises("mask must be uint8 or bool", fn, lg, idx, mask=torch.zeros(4))
        _raises("logits must be a device", fn, lg, idx)
    _raises("idx: shape", bf.group_pairs, idx[0], 8)
    _raises(r"offsets: shape \(9,\)", bf.group_pairs, idx, 8, offsets=torch.zeros(8, dtype=torch.int32))
