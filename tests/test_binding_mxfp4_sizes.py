"""Host checks (no GPU) of the sizes and numbers that the 4-bit float, grouping
and router-loss calls hand to the library as 32-bit integers: one that does not
fit is refused, never cut to its low bits."""
import pytest
import torch

bf = pytest.importorskip("bit_expert_ffn_top_amd")

BIG = 1 << 32
I32 = dict(dtype=torch.int32)


def _raises(match, fn, *a, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


def _meta(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")   # a shape without memory


def _q(*shape, make=torch.zeros, **kw):
    return bf.Mxfp4(make(shape[:-1] + (shape[-1] // 2,), dtype=torch.uint8, **kw),
                    make(shape[:-1] + (shape[-1] // 32,), dtype=torch.uint8, **kw))


def _meta_q(*shape):
    return _q(*shape, make=torch.empty, device="meta")


@pytest.mark.parametrize("value", [BIG + 1, BIG, 1 << 31, -(1 << 31) - 1, 2.5])
def test_numbers(value):
    """2^32 + 1 would become 1, 2^32 the first slot, 2.5 a divisor of 2."""
    for fn in (bf.mxfp4_linear, bf.mxfp4_gate_up):
        _raises("src_div: a 32-bit integer", fn, _q(4, 64), _q(64, 64), src_div=value)
    _raises("shared_slot: a 32-bit integer", bf.mxfp4_ffn_decode, _q(4, 64, 64), _q(4, 64, 32), torch.zeros(2, 64),
            torch.zeros((2, 3), **I32), torch.zeros(2, 3), shared_slot=value)
    _raises("n_experts: a 32-bit integer", bf.group_pairs, torch.zeros((4, 2), **I32), value)


@pytest.mark.parametrize("n", [BIG + 4, 1 << 31])
def test_extents(n):
    _raises("32-bit", bf.mxfp4_quantize, _meta(1, n - n % 32 + 64))
    _raises("32-bit", bf.mxfp4_dequantize, _meta_q(1, n - n % 32 + 64))
    for fn in (bf.mxfp4_linear, bf.mxfp4_gate_up):
        _raises("32-bit", fn, _q(4, 64), _meta_q(n - n % 64 + 64, 64))
        _raises("32-bit", fn, _meta_q(n, 64), _q(64, 64))
    _raises("32-bit", bf.group_pairs, _meta(n, 1, dtype=torch.int32), 8)
    _raises("32-bit", bf.mxfp4_ffn_decode, _q(4, 64, 64), _q(4, 64, 32), _meta(n, 64), _meta(n, 1, dtype=torch.int32),
            _meta(n, 1))
    _raises("32-bit", bf.mxfp4_ffn_decode, _q(4, 64, 64), _q(4, 64, 32), _meta(1, 64), _meta(1, n, dtype=torch.int32),
            _meta(1, n))
    for fn in (bf.route_balance, bf.route_backward):
        _raises("32-bit", fn, _meta(n, 8), _meta(n, 2, dtype=torch.int32))
        _raises("32-bit", fn, _meta(4, n), _meta(4, 2, dtype=torch.int32))
        _raises("32-bit", fn, _meta(4, 8), _meta(4, n, dtype=torch.int32))
        _raises("32-bit", fn, _meta(4, 8), _meta(4, 2, dtype=torch.int32), seq_offsets=_meta(n + 1, dtype=torch.int32))


@pytest.mark.parametrize("fn,args", [(bf.group_workspace_bytes, (100, 8)), (bf.route_balance_workspace_bytes, (100, 8, 3)),
                                     (bf.mxfp4_ffn_decode_workspace_bytes, (4, 10, 64))])
def test_workspace_sizes(fn, args):
    try:
        bf.lib()
    except RuntimeError as e:
        pytest.skip(str(e))
    assert fn(*args) > 0
    for i in range(len(args)):
        _raises("32-bit integer", fn, *args[:i], args[i] + BIG, *args[i + 1:])


def test_numbers_that_fit_pass():
    """The check before the devices lets ordinary numbers on, of any integer type."""
    import numpy as np
    for value in (1, np.int64(3), torch.tensor(2), 4.0, (1 << 31) - 1):
        _raises("a.codes must be a device tensor", bf.mxfp4_linear, _q(4, 64), _q(64, 64), src_div=value)
