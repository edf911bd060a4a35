"""Host checks (no GPU) of the dispatch to the experts and back, the adapters and
the verification of drafted tokens: the C entry points refuse bad arguments
before any HIP call, the binding refuses wrong shapes, types, sizes and places
before the library."""
import ctypes
import itertools

import pytest
import torch

bf = pytest.importorskip("bit_expert_ffn_top_amd")

BASE = 0x7F0000000000  # never dereferenced: every call below fails its host checks
EINVAL, EALIGN, ENOSPC = -1, -2, -4
BIG, INT_MAX, INT_MIN = 1 << 32, (1 << 31) - 1, -(1 << 31)
I32 = dict(dtype=torch.int32)


def _lib():
    try:
        return bf.lib()
    except RuntimeError as e:
        pytest.skip(str(e))


def _at(i, off=0):
    return ctypes.c_void_p(BASE + (i << 32) + off)


def _dispatch(p, dtype=1, T=100, d=64, k=2, E=8, nb=1 << 30):
    return _lib().moe_dispatch(p["x"], dtype, T, d, p["idx"], k, E, p["rows"], p["offsets"], p["pair_pos"], p["ws"], nb,
                               None)


def _combine(p, rt=1, R=200, T=100, d=64, k=2, bt=1, yt=1):
    return _lib().moe_combine_rows(p["rows"], rt, R, T, d, k, p["pair_pos"], p["w"], p["base"], bt, p["y"], yt, None)


def _backward(p, gt=1, rt=1, R=200, T=100, d=64, k=2):
    return _lib().moe_combine_backward(p["dy"], gt, p["rows"], rt, R, T, d, k, p["pair_pos"], p["w"], p["drows"],
                                       p["dw"], None)


def _lora(p, xt=1, T=100, d_in=64, d_out=48, n=4, rank=16, S=7, yt=1, nb=1 << 40):
    return _lib().moe_lora(p["base"], p["x"], xt, T, d_in, d_out, p["a"], p["b"], n, rank, p["seq"], S, p["adapter"],
                           p["scale"], p["y"], yt, p["ws"], nb, None)


def _verify(p, dtype=0, B=3, n=4, V=1000, nb=1 << 30):
    return _lib().moe_verify_drafts(p["p"], p["q"], dtype, B, n, V, p["draft"], p["n_draft"], p["ua"], p["us"],
                                    p["tokens"], p["n_accepted"], p["ws"], nb, None)


# call -> (what it writes, what it reads, which of these may be null)
CALLS = {
    _dispatch: (["rows", "offsets", "pair_pos"], ["x", "idx"], []),
    _combine: (["y"], ["rows", "pair_pos", "w", "base"], ["w", "base"]),
    _backward: (["drows", "dw"], ["dy", "rows", "pair_pos", "w"], ["w", "drows", "dw"]),
    _lora: (["y"], ["x", "base", "a", "b", "seq", "adapter", "scale"], ["seq", "scale"]),
    _verify: (["tokens", "n_accepted"], ["p", "q", "draft", "n_draft", "ua", "us"], ["q", "n_draft"]),
}


def _ptrs(call):
    names = CALLS[call][0] + CALLS[call][1] + ["ws"]
    return {n: _at(i) for i, n in enumerate(names)}


EACH = [(c, n) for c, (w, r, _) in CALLS.items() for n in w + r]


def _ids(v):
    return v.__name__.strip("_") if callable(v) else str(v)


@pytest.mark.parametrize("call,name", EACH, ids=_ids)
def test_null_and_misaligned(call, name):
    p = _ptrs(call)
    written, read, may = CALLS[call]
    if name not in may:
        assert call({**p, name: None}) == EINVAL
    i = (written + read).index(name)
    for off in (1, 2, 4, 8):
        assert call({**p, name: _at(i, off)}) == EALIGN


PAIRS = [(c, a, b) for c, (w, r, _) in CALLS.items()
         for a, b in itertools.chain(itertools.combinations(w, 2), itertools.product(w, r))
         if (c, a, b) != (_lora, "y", "base")]      # the results may take base's place


@pytest.mark.parametrize("call,a,b", PAIRS, ids=_ids)
def test_one_buffer_twice(call, a, b):
    if (a, b) == ("y", "base"):
        assert call({**_ptrs(call), a: _at(9), b: _at(9)}, bt=0) == EINVAL     # base's place, but not its type
        return
    assert call({**_ptrs(call), a: _at(9), b: _at(9)}) == EINVAL


def test_both_gradients_missing():
    assert _backward({**_ptrs(_backward), "drows": None, "dw": None}) == EINVAL


def test_sizes():
    for call in (_dispatch, _combine, _backward):
        p = _ptrs(call)
        most = 65536 if call is _dispatch else (1 << 24) - 1
        for T in (-1, most + 1, INT_MAX, INT_MIN):
            assert call(p, T=T) == EINVAL, T
        for k in (0, -1, 65, INT_MAX):
            assert call(p, k=k) == EINVAL, k
        for d in (0, -4, 2, 6, 16384 + 4, INT_MAX, INT_MIN):
            assert call(p, d=d) == EINVAL, d
    for E in (0, -1, 1025, INT_MAX):
        assert _dispatch(_ptrs(_dispatch), E=E) == EINVAL
    for call in (_combine, _backward):
        for R in (-1, 1 << 31, (1 << 63) - 1, -(1 << 63)):
            assert call(_ptrs(call), R=R) == EINVAL
        assert call({n: None for n in _ptrs(call)}, T=0) == 0
    p = _ptrs(_lora)
    for T in (-1, 1 << 24, (1 << 63) - 1):
        assert _lora(p, T=T) == EINVAL
    for d in (0, -32, 16, 48, 16384 + 32, INT_MAX):
        assert _lora(p, d_in=d) == EINVAL
    for d in (0, -16, 8, 24, 16384 + 16, INT_MAX):
        assert _lora(p, d_out=d) == EINVAL
    for n in (0, -1, 1025, INT_MAX):
        assert _lora(p, n=n) == EINVAL
    for r in (0, -8, 4, 12, 136, INT_MAX):
        assert _lora(p, rank=r) == EINVAL
    for S in (0, -1, 65537, INT_MAX):
        assert _lora(p, S=S) == EINVAL
    assert _lora({**p, "seq": None}) == EINVAL            # seven requests, 100 rows
    assert _lora({n: None for n in p}, T=0, S=0) == 0
    p = _ptrs(_verify)
    for B in (-1, 65537, INT_MAX, INT_MIN):
        assert _verify(p, B=B) == EINVAL
    for n in (-1, 64, INT_MAX):
        assert _verify(p, n=n) == EINVAL
    for V in (0, -1, 1 << 24, INT_MAX):
        assert _verify(p, V=V) == EINVAL
    assert _verify({n: None for n in p}, B=0) == 0


def test_types():
    for t in (-1, 2, 7):
        assert _dispatch(_ptrs(_dispatch), dtype=t) == EINVAL
        assert _verify(_ptrs(_verify), dtype=t) == EINVAL
        for name in ("rt", "bt", "yt"):
            assert _combine(_ptrs(_combine), **{name: t}) == EINVAL
        for name in ("gt", "rt"):
            assert _backward(_ptrs(_backward), **{name: t}) == EINVAL
        for name in ("xt", "yt"):
            assert _lora(_ptrs(_lora), **{name: t}) == EINVAL


def test_workspaces():
    """Where a call needs a workspace, a missing, short or misaligned one, or one
    that is another of its buffers, is refused; sizes out of range need none."""
    lib = _lib()
    for bad in ((-1, 2, 8), (65537, 2, 8), (8, 0, 8), (8, 65, 8), (8, 2, 0), (8, 2, 1025), (INT_MAX, INT_MAX, INT_MAX)):
        assert lib.moe_dispatch_workspace_bytes(*bad) == 0, bad
    for bad in ((-1, 10), (65537, 10), (1, 0), (1, 1 << 24), (INT_MAX, INT_MAX)):
        assert lib.moe_verify_drafts_workspace_bytes(*bad) == 0, bad
    for bad in ((-1, 16, 4), (1 << 24, 16, 4), (9999, 12, 4), (9999, 136, 4), (9999, 16, -1), (9999, 16, 65537)):
        assert lib.moe_lora_workspace_bytes(*bad) == 0, bad
    cases = [(_lora, lib.moe_lora_workspace_bytes(1 << 20, 128, 7), dict(T=1 << 20, rank=128)),
             (_dispatch, lib.moe_dispatch_workspace_bytes(60000, 64, 1000), dict(T=60000, k=64, E=1000)),
             (_verify, lib.moe_verify_drafts_workspace_bytes(1, 1 << 20), dict(B=1, V=1 << 20))]
    for call, need, kw in cases:
        p = _ptrs(call)
        if need:
            i = len(CALLS[call][0] + CALLS[call][1])
            assert call({**p, "ws": None}, **kw) == EINVAL
            assert call({**p, "ws": _at(i, 128)}, **kw) == EALIGN
            assert call(p, nb=need - 1, **kw) == ENOSPC
            for name in CALLS[call][0] + CALLS[call][1]:
                assert call({**p, "ws": p[name]}, **kw) == EINVAL


# --- the binding ----------------------------------------------------------------


def _raises(match, fn, *a, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


def _meta(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")   # a shape without memory


def test_binding_dispatch():
    x, idx = torch.zeros(5, 8), torch.zeros((5, 2), **I32)
    _raises("x must be float32 or bfloat16", bf.dispatch, x.half(), idx, 4)
    _raises("x: shape", bf.dispatch, x[0], idx, 4)
    _raises("idx: shape", bf.dispatch, x, idx[:4], 4)
    _raises(r"rows: shape \(10, 8\)", bf.dispatch, x, idx, 4, rows=torch.zeros(9, 8))
    _raises(r"offsets: shape \(5,\)", bf.dispatch, x, idx, 4, offsets=torch.zeros(4, **I32))
    _raises(r"pair_pos: shape \(5, 2\)", bf.dispatch, x, idx, 4, pair_pos=torch.zeros((2, 5), **I32))
    _raises("x must be a device tensor", bf.dispatch, x, idx, 4)
    for n in (BIG + 1, 2.5):
        _raises("n_experts: a 32-bit integer", bf.dispatch, x, idx, n)
    _raises("32-bit", bf.dispatch, _meta(BIG + 1, 8), _meta(BIG + 1, 2, **I32), 4)
    _raises("32-bit", bf.dispatch, _meta(1 << 30, 8), _meta(1 << 30, 2, **I32), 4)


def test_binding_combine():
    rows, pos, w = torch.zeros(10, 8), torch.zeros((5, 2), **I32), torch.zeros(5, 2)
    _raises("rows must be float32 or bfloat16", bf.combine_rows, rows.double(), pos)
    _raises("rows: shape", bf.combine_rows, rows[0], pos)
    _raises("pair_pos: shape", bf.combine_rows, rows, pos[0])
    _raises("w: shape", bf.combine_rows, rows, pos, w[:4])
    _raises(r"base: shape \(5, 8\)", bf.combine_rows, rows, pos, base=torch.zeros(5, 4))
    _raises("base must be float32 or bfloat16", bf.combine_rows, rows, pos, base=torch.zeros(5, 8).half())
    _raises(r"y: shape \(5, 8\)", bf.combine_rows, rows, pos, y=torch.zeros(5, 4))
    _raises("y must be float32 or bfloat16", bf.combine_rows, rows, pos, dtype=torch.float16)
    _raises("rows must be a device tensor", bf.combine_rows, rows, pos)
    _raises(r"y: shape \(5, 8\)", bf.dispatch_backward, rows, pos, dx=torch.zeros(5, 4))
    _raises("32-bit", bf.combine_rows, _meta(BIG, 8), pos)


def test_binding_combine_backward():
    dy, rows, pos, w = torch.zeros(5, 8), torch.zeros(10, 8), torch.zeros((5, 2), **I32), torch.zeros(5, 2)
    f = bf.combine_backward
    _raises("dy must be float32 or bfloat16", f, dy.half(), rows, pos)
    _raises("rows must be float32 or bfloat16", f, dy, rows.half(), pos)
    _raises("dy: shape", f, dy[0], rows, pos)
    _raises(r"rows: shape \(\*, 8\)", f, dy, torch.zeros(10, 4), pos)
    _raises("pair_pos: shape", f, dy, rows, pos[:4])
    _raises("rows must be a device tensor", f, dy, rows, pos, w)
    _raises("rows: expected where dw", f, dy, None, pos, w, drows=rows)
    _raises("rows, or drows", f, dy, None, pos, w, need_w=False)
    _raises("must be needed", f, dy, rows, pos, w, need_rows=False, need_w=False)
    _raises("not needed", f, dy, rows, pos, w, drows=rows, need_rows=False)
    _raises("not needed", f, dy, rows, pos, w, dw=w, need_w=False)
    _raises("drows: shape", f, dy, rows, pos, w, drows=torch.zeros(9, 8))


def test_binding_lora():
    base, x = torch.zeros(5, 48), torch.zeros(5, 64)
    a, b = torch.zeros((3, 16, 64), dtype=torch.bfloat16), torch.zeros((3, 48, 16), dtype=torch.bfloat16)
    who = torch.zeros(5, **I32)
    _raises("x must be float32 or bfloat16", bf.lora, base, x.half(), a, b, who)
    _raises("base must be float32 or bfloat16", bf.lora, base.half(), x, a, b, who)
    _raises("base: shape", bf.lora, base[:4], x, a, b, who)
    _raises(r"a: shape \(\*, \*, 64\)", bf.lora, base, x, a[..., :32], b, who)
    _raises(r"b: shape \(3, 48, 16\)", bf.lora, base, x, a, b[:2], who)
    _raises(r"adapter: shape \(5,\)", bf.lora, base, x, a, b, who[:4])
    _raises(r"seq_offsets: shape \(6,\)", bf.lora, base, x, a, b, who, seq_offsets=torch.zeros(5, **I32))
    _raises("scale must be a device tensor", bf.lora, base, x, a, b, who, scale=torch.zeros(3))
    _raises(r"scale: shape \(3,\)", bf.lora, base, x, a, b, who, scale=torch.zeros(2))
    _raises(r"y: shape \(5, 48\)", bf.lora, base, x, a, b, who, y=torch.zeros(5, 32))
    _raises("x must be a device tensor", bf.lora, base, x, a, b, who)
    _raises("32-bit", bf.lora, _meta(BIG, 48), _meta(BIG, 64), a, b, _meta(BIG, **I32))


def test_binding_verify():
    p, q, draft = torch.zeros(3, 5, 100), torch.zeros(3, 4, 100), torch.zeros((3, 4), **I32)
    ua, us = torch.zeros(3, 4), torch.zeros(3)
    f = bf.verify_drafts
    _raises("p must be float32 or bfloat16", f, p.half(), q, draft, ua, us)
    _raises(r"p: shape \(3, 5, \*\)", f, p[:, :4], q, draft, ua, us)
    _raises("q must be a device tensor", f, p, q.bfloat16(), draft, ua, us)
    _raises(r"q: shape \(3, 4, 100\)", f, p, q[:, :3], draft, ua, us)
    _raises("draft: shape", f, p, q, draft[0], ua, us)
    _raises("at most 63 drafts", f, torch.zeros(1, 65, 4), None, torch.zeros((1, 64), **I32), ua, us)
    _raises("u_accept: shape", f, p, None, draft, ua[:, :3], us)
    _raises("u_accept must be a device tensor", f, p, None, draft, ua, us)
    _raises("32-bit", f, _meta(3, 5, BIG), None, draft, ua, us)
