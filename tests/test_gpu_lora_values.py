"""GPU tests of values that a product of parts can get wrong: infinities and NaN of
x, values of h that cancel.  Every form of the call: few rows, many rows, and both of
gathered rows.
"""
import numpy as np
import pytest
import torch

import oracle.lora as ol
from parity import need_gpu
from test_gpu_lora import BF16, F32, TYPES, _bf, _bound, _i32, _inputs, _np

pytestmark = pytest.mark.gpu

# rows, bounds of the requests (None: a row for each)
FORMS = {"few": (20, [0, 12, 20]), "gathered": (200, None), "many": (1100, [0, 600, 1100]),
         "many gathered": (1600, None)}


def _form(name):
    """(T, bounds, the adapter of every request, that of every row), two adapters."""
    T, seq = FORMS[name]
    who = np.arange(T if seq is None else len(seq) - 1) % 2
    return T, seq, who, who if seq is None else np.repeat(who, np.diff(seq))


def _call(form, base, x, a, b, scale=None):
    _, seq, who, _ = _form(form)
    return _bf().lora(base, x, a, b, _i32(who), seq_offsets=None if seq is None else _i32(seq), scale=scale)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("form", FORMS)
def test_infinities_are_the_formulas(form, types):
    """An infinity in x gives the infinities and NaN that the formula gives in 64
    bits, whatever parts its type enters as: a column of A of one sign, rows of B of
    one sign (infinite results) and of both (NaN), infinities of both signs in a row,
    an infinity times zero, a NaN whose high half is an infinity's."""
    T, seq, who, of = _form(form)
    base, x, a, b, scale = _inputs(T, 2, 16, 96, 48, *types)
    a[:, :, 13] = a[:, :, 13].abs() + 0.5
    a[:, :, 70] = a[:, :, 70].abs() + 0.5
    a[1, 3, 70] = 0.0
    sign = 1.0 - 2.0 * (torch.arange(44, device=b.device) % 2)
    b[:, :44] = ((b[:, :44].abs() + 0.25) * sign[None, :, None]).to(BF16)
    inf = float("inf")
    rows = [1, 2, 13, 14, T // 2 + 2, T // 2 + 3, T - 2, T - 1]
    for i, t in enumerate(rows):
        if i % 4 < 3:
            x[t, 13] = (inf, -inf, inf)[i % 4]
        if i % 4 == 2:
            x[t, 70] = -inf
        if i % 4 == 3:
            x[t, 70] = inf
    low = 5
    if x.dtype == F32:
        x.view(torch.int32)[low, 20] = 0x7F800001
    else:
        x[low, 20] = float("nan")
    got = _np(_call(form, base, x, a, b, scale))
    with np.errstate(invalid="ignore"):
        r = ol.lora(_np(base), _np(x), _np(a), _np(b), who, seq, _np(scale))
    special = np.zeros(T, bool)
    special[rows + [low]] = True
    want = r["y"]
    assert not np.isfinite(want[special]).any() and np.isinf(want[special]).any() and np.isnan(want[low]).all()
    assert np.array_equal(got[special], want[special], equal_nan=True)
    with np.errstate(invalid="ignore"):
        ok = np.abs(got - want) <= _bound(r, 96, 16, base.dtype)
    assert ok[~special].all()


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("form", FORMS)
def test_values_of_h_that_cancel(form, types):
    """Two ranks whose h differ by one value of x and whose columns of B are opposite:
    y is that value times B's.  All values are whole numbers: h between 2^18 and
    2^20, sums of both products below 2^24, and y of at most 254, so that fp32 sums
    and one rounding to the output's type are exact, and any bit of h that is lost is
    seen."""
    T, _, _, of = _form(form)
    xt, yt = types
    dev = need_gpu()
    g = torch.Generator().manual_seed(T)
    x = torch.randint(64, 128, (T, 64), generator=g) * (1 - 2 * torch.randint(0, 2, (T, 1), generator=g))
    x = x.to(xt).to(dev)
    a = torch.zeros((2, 16, 64))
    a[:, 2] = torch.randint(64, 127, (2, 64), generator=g).float()
    a[:, 9] = a[:, 2]
    a[0, 9, 40] += 1
    a[1, 9, 7] += 1
    b = torch.zeros((2, 48, 16))
    c = (torch.arange(48) % 2 + 1).float()
    b[:, :, 2], b[:, :, 9] = -c, c
    a, b = a.to(BF16).to(dev), b.to(BF16).to(dev)
    y = _call(form, torch.zeros((T, 48), dtype=yt, device=dev), x, a, b)
    at = torch.from_numpy(np.where(of == 0, 40, 7)).to(dev)
    want = x.float().gather(1, at[:, None]) * c.to(dev)
    assert torch.equal(y.float(), want)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("form", FORMS)
def test_h_past_the_largest_bfloat16(form, types):
    """A finite h that lies between the largest bfloat16 and the largest fp32 value is
    no infinity: h = x0 + x1, a sum that fp32 holds exactly, times a power of two,
    rounded once."""
    T, _, _, of = _form(form)
    xt, yt = types
    dev = need_gpu()
    top = 2.0 ** 127 * (2 - 2.0 ** -7)             # the largest bfloat16
    x = torch.zeros((T, 64))
    x[:, 5], x[:, 60] = top, 2.0 ** 119 + 2.0 ** 113 * (torch.arange(T) % 2)
    x = (x * (1 - 2 * (torch.arange(T) % 3 == 1).float())[:, None]).to(xt)
    a, b = torch.zeros((2, 16, 64)), torch.zeros((2, 48, 16))
    a[:, 11, 5] = a[:, 11, 60] = 1.0
    p = 2.0 ** -(torch.arange(48) % 7 + 3.0)
    b[0, :, 11], b[1, :, 11] = p, -p
    h = x[:, 5].double() + x[:, 60].double()
    assert (h.abs() > top + 2.0 ** 118).all() and torch.equal(h.float().double(), h)
    sign = torch.from_numpy(np.where(of == 0, 1.0, -1.0))
    want = (sign[:, None] * h[:, None] * p.double()).to(yt)
    y = _call(form, torch.zeros((T, 48), dtype=yt, device=dev), x.to(dev), a.to(BF16).to(dev), b.to(BF16).to(dev))
    assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("yt", [F32, BF16])
@pytest.mark.parametrize("rank", [8, 32, 40, 64, 72, 128])
@pytest.mark.parametrize("form", ["many", "many gathered"])
def test_a_workspace_of_the_size_that_is_asked_for(form, rank, yt):
    """Nothing is written past it, and it may hold anything."""
    bf = _bf()
    T, seq, who, _ = _form(form)
    base, x, a, b, scale = _inputs(T, 2, rank, 96, 48, BF16, yt)
    want = _call(form, base, x, a, b, scale)
    need = bf.lora_workspace_bytes(T, rank, 0 if seq is None else len(who))
    assert need > 0
    ws = torch.full((need + 65536,), 0xFF, dtype=torch.uint8, device=x.device)
    y = bf.lora(base, x, a, b, _i32(who), seq_offsets=None if seq is None else _i32(seq), scale=scale, ws=ws[:need])
    assert torch.equal(y, want) and (ws[need:] == 0xFF).all()
