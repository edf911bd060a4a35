"""GPU tests of the calls of a step for many requests together: a batched verify
step with adapters and its gradients, side streams, replayed graphs, refusals on
the device.  Bars: those of test_gpu_dispatch, test_gpu_lora and
test_gpu_verify_drafts, applied to each call's own inputs.
"""
import numpy as np
import pytest
import torch

import oracle.dispatch as od
import oracle.drafts as odr
import oracle.lora as ol
from parity import need_gpu
from test_gpu_dispatch import HALF_STEP, U, _bf, _np
from test_gpu_lora import _bound, _i32

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _layer(seed, R=5, drafts=3, E=16, k=4, d=256, F=64, V=20000, n=3, rank=16):
    """Inputs of a verify step of R requests with 1 + drafts tokens each."""
    bf = _bf()
    dev = need_gpu()
    g = torch.Generator().manual_seed(seed)

    def randn(*shape, scale=1.0, dtype=F32):
        return (torch.randn(shape, generator=g) * scale).to(dtype).to(dev)

    T = R * (drafts + 1)
    s = dict(E=E, k=k, x=randn(T, d), logits=randn(T, E, scale=1.5), seq=_i32(np.arange(R + 1) * (drafts + 1)),
             adapter=_i32(np.arange(R) % (n + 1) - 1), scale=0.5 + torch.rand((n,), generator=g).to(dev),
             a=randn(n, rank, d, scale=d ** -0.5, dtype=BF16), b=randn(n, 2 * F, rank, scale=rank ** -0.5, dtype=BF16),
             gate_up=bf.mxfp4_quantize(randn(E, 2 * F, d, scale=d ** -0.5)),
             down=bf.mxfp4_quantize(randn(E, d, F, scale=F ** -0.5)),
             shared_gate_up=bf.mxfp4_quantize(randn(2 * F, d, scale=d ** -0.5)),
             shared_down=bf.mxfp4_quantize(randn(d, F, scale=F ** -0.5)),
             head=randn(d, V, scale=d ** -0.5), q=torch.softmax(randn(R, drafts, V), -1),
             draft=torch.randint(0, V, (R, drafts), generator=g).int().to(dev),
             ua=torch.rand((R, drafts), generator=g).to(dev), us=torch.rand((R,), generator=g).to(dev),
             dy=randn(T, d))
    return s


def _step(s):
    """The step; every call's results."""
    bf = _bf()
    x, R = s["x"], s["draft"].shape[0]
    idx, w = bf.route_topk(s["logits"], s["k"])
    f = bf.dispatch(x.bfloat16(), idx, s["E"], rows=torch.zeros((idx.numel(), x.shape[1]), dtype=BF16, device=x.device))
    h = bf.mxfp4_gate_up(bf.mxfp4_quantize(f.rows), s["gate_up"], f.offsets)
    rows = bf.mxfp4_linear(bf.mxfp4_quantize(h), s["down"], f.offsets, dtype=BF16)
    proj = bf.mxfp4_linear(bf.mxfp4_quantize(x), s["shared_gate_up"])
    gu = bf.lora(proj, x, s["a"], s["b"], s["adapter"], seq_offsets=s["seq"], scale=s["scale"])
    hs = torch.nn.functional.silu(gu[:, 0::2]) * gu[:, 1::2]
    base = x + bf.mxfp4_linear(bf.mxfp4_quantize(hs), s["shared_down"])
    y = bf.combine_rows(rows, f.pair_pos, w, base=base, dtype=F32)
    p = torch.softmax(y @ s["head"], -1).view(R, -1, s["head"].shape[1])
    q = torch.where(s["ua"][..., None] < 0.5, s["q"], p[:, :-1]).contiguous()   # some drafters agree with the target
    tokens, accepted = bf.verify_drafts(p, q, s["draft"], s["ua"], s["us"])
    drows, dw = bf.combine_backward(s["dy"], rows, f.pair_pos, w, drows=torch.zeros_like(rows))
    dlogits = bf.route_backward(s["logits"], idx, w=w, dw=dw)
    dx = bf.dispatch_backward(drows, f.pair_pos, dtype=F32)
    return dict(idx=idx, w=w, rows_in=f.rows, offsets=f.offsets, pair_pos=f.pair_pos, rows=rows, proj=proj, gu=gu,
                base=base, y=y, p=p, q=q, tokens=tokens, accepted=accepted, drows=drows, dw=dw, dlogits=dlogits, dx=dx)


def test_a_verify_step_of_many_requests():
    s = _layer(1)
    r = _step(s)
    idx = r["idx"].cpu().numpy()
    offsets, pos = od.positions(idx, s["E"])
    assert np.array_equal(r["offsets"].cpu().numpy(), offsets) and np.array_equal(r["pair_pos"].cpu().numpy(), pos)
    xb = s["x"].bfloat16()
    for t in range(xb.shape[0]):
        assert torch.equal(r["rows_in"][torch.from_numpy(pos[t]).to(xb.device)], xb[t].expand(s["k"], -1))
    ref, mag = od.combine_rows(_np(r["rows"]), pos, _np(r["w"]), _np(r["base"]))
    assert (np.abs(_np(r["y"]) - ref) <= (s["k"] + 2) * U * mag + U * np.abs(ref)).all()
    la = ol.lora(_np(r["proj"]), _np(s["x"]), _np(s["a"]), _np(s["b"]), s["adapter"].cpu().numpy(),
                 s["seq"].cpu().numpy(), _np(s["scale"]))
    assert (np.abs(_np(r["gu"]) - la["y"]) <= _bound(la, s["x"].shape[1], 16, F32)).all()
    tokens, count = odr.verify(r["p"].cpu().numpy(), r["q"].cpu().numpy(), s["draft"].cpu().numpy(),
                               s["ua"].cpu().numpy(), s["us"].cpu().numpy())
    assert np.array_equal(r["tokens"].cpu().numpy(), tokens) and np.array_equal(r["accepted"].cpu().numpy(), count)


def test_gradients_through_the_routing_weights():
    """dlogits and dx against autograd in 64 bits over the same choice: y = base +
    sum of softmax(chosen logits) times the rows, which stand still for dlogits;
    and rows that are x itself for dx.  dw is off by (d + 2) u mag, and dlogits =
    w (dw - sum w dw) by w (that + its weighted mean) and 6 roundings of terms of
    size w (|dw| + sum w |dw|)."""
    s = _layer(2)
    r = _step(s)
    T, k, d = s["x"].shape[0], s["k"], s["x"].shape[1]
    idx, pos = r["idx"].cpu().long(), r["pair_pos"].cpu().long()
    lg = s["logits"].double().cpu().requires_grad_()
    w = torch.softmax(lg.gather(1, idx), 1)
    rows = r["rows"].double().cpu()
    ((w[..., None] * rows[pos]).sum(1) * s["dy"].double().cpu()).sum().backward()
    _, dw, mag = od.combine_backward(_np(s["dy"]), _np(r["rows"]), pos.numpy(), None)
    w = w.detach().numpy()
    ddw = (d + 2) * U * mag
    err = w * (ddw + (w * ddw).sum(1, keepdims=True)) + 16 * U * w * (np.abs(dw) + (w * np.abs(dw)).sum(1, keepdims=True))
    full = np.zeros((T, s["E"]))
    np.put_along_axis(full, idx.numpy(), err, 1)
    assert (np.abs(_np(r["dlogits"]) - lg.grad.numpy()) <= full).all()
    # dx: each row's gradient is bf16(w dy), and the sum of the k of them in fp32
    wg = r["w"].double().cpu()
    g = (wg[..., None] * s["dy"].double().cpu()[:, None]).numpy()
    bar = (HALF_STEP[BF16] * (1 + U) + U) * np.abs(g).sum(1) + (k + 2) * U * np.abs(g).sum(1) * 1.01
    assert (np.abs(_np(r["dx"]) - g.sum(1)) <= bar).all()


def test_streams_and_graphs():
    """The step on a side stream and in a graph replayed with other inputs between
    eager steps: always the eager bits."""
    bf = _bf()
    sets = [_layer(i) for i in (3, 4, 5)]
    eager = [_step(s) for s in sets]
    torch.cuda.synchronize()
    live = {n: (v.clone() if torch.is_tensor(v) else v) for n, v in sets[0].items()}
    fixed = ("gate_up", "down", "shared_gate_up", "shared_down")
    for n in fixed:
        live[n] = bf.Mxfp4(live[n].codes.clone(), live[n].scales.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = _step(live)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(there[n], eager[0][n]) for n in there)
    graph = torch.cuda.CUDAGraph()
    names = [n for n, v in live.items() if torch.is_tensor(v)]
    with torch.cuda.graph(graph):
        got = _step(live)
    for i in (1, 2, 0, 1, 2):
        for n in names:
            live[n].copy_(sets[i][n])
        for n in fixed:
            live[n].codes.copy_(sets[i][n].codes)
            live[n].scales.copy_(sets[i][n].scales)
        graph.replay()
        torch.cuda.synchronize()
        again = _step(sets[i])
        for n in got:
            assert torch.equal(again[n], eager[i][n]), (i, n)
            assert torch.equal(got[n], eager[i][n]), (i, n)


def test_large_calls_on_a_stream_of_their_own_and_in_one_graph():
    """The variants for many tokens, rows and long rows, two calls of each with
    workspaces of their own in one graph, and given a stream while another one is
    the current one."""
    bf = _bf()
    dev = need_gpu()
    g = torch.Generator().manual_seed(9)
    T, k, E, d = 3000, 8, 100, 64
    idx = [torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int().to(dev) for _ in range(2)]
    x = [torch.randn((T, d), generator=g).bfloat16().to(dev) for _ in range(2)]
    a = torch.randn((3, 16, d), generator=g).bfloat16().to(dev)
    b = torch.randn((3, 32, 16), generator=g).bfloat16().to(dev)
    base = torch.randn((T, 32), generator=g).bfloat16().to(dev)
    seq, who = _i32([0, 1000, 1001, T]), _i32([2, 0, 1])
    p = torch.softmax(torch.randn((4, 3, 40000), generator=g), -1).to(dev)
    draft = torch.randint(0, 40000, (4, 2), generator=g).int().to(dev)
    ua, us = torch.full((4, 2), 1e-6, device=dev), torch.rand((4,), generator=g).to(dev)

    def calls(stream=None):
        out = []
        for i in range(2):
            f = bf.dispatch(x[i], idx[i], E, stream=stream)
            out += [*f, bf.lora(base, x[i], a, b, who, seq_offsets=seq, stream=stream),
                    *bf.verify_drafts(p, None, draft, ua, us, stream=stream)]
        return out

    want = calls()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = calls(side)
    side.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got, want))
        calls()


def test_device_refusals():
    bf = _bf()
    dev = need_gpu()
    x, idx = torch.randn((6, 8), device=dev), _i32([[0, 1]] * 6)
    with pytest.raises(ValueError, match="contiguous"):
        bf.dispatch(x.t().contiguous().t(), idx, 4)
    with pytest.raises(ValueError, match="x must be a device tensor"):
        bf.dispatch(x.cpu(), idx, 4)
    with pytest.raises(ValueError, match="idx must be torch.int32"):
        bf.dispatch(x, idx.long(), 4)
    with pytest.raises(bf.MoeError, match="invalid argument"):
        bf.dispatch(x[:, :6].contiguous(), idx, 4)                       # six columns
    with pytest.raises(bf.MoeError, match="misaligned"):
        bf.combine_rows(torch.zeros((100,), device=dev)[1:65].view(8, 8), idx)
    with pytest.raises(bf.MoeError, match="invalid argument"):
        bf.combine_rows(x, idx[:, :1].contiguous(), y=x)                  # in the rows' place
    with pytest.raises(bf.MoeError, match="invalid argument"):
        bf.combine_backward(torch.ones_like(x), x, idx[:, :1].contiguous(), drows=x)
    big = torch.zeros((9000, 8), device=dev)
    with pytest.raises(bf.MoeError, match="workspace"):
        bf.dispatch(big, _i32(np.zeros((9000, 1))), 4, ws=torch.empty((255,), dtype=torch.uint8, device=dev))
    p = torch.rand((1, 2, 30000), device=dev)
    with pytest.raises(bf.MoeError, match="workspace"):
        bf.verify_drafts(p, None, _i32([[1]]), torch.rand((1, 1), device=dev), torch.rand((1,), device=dev),
                         ws=torch.empty((64,), dtype=torch.uint8, device=dev))
    a, b = torch.zeros((2, 12, 32), dtype=BF16, device=dev), torch.zeros((2, 16, 12), dtype=BF16, device=dev)
    with pytest.raises(bf.MoeError, match="invalid argument"):            # rank 12
        bf.lora(torch.zeros((6, 16), device=dev), torch.zeros((6, 32), device=dev), a, b, _i32([0] * 6))
