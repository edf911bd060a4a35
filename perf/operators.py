"""The operators measured in this repository, with their plain forms.

Five operators that stand beside the routed-expert FFN over packed experts:

  quantize    rows of fp32 or bf16 values to microscaled 4-bit floats (blocks
              of 32 values, one power-of-two scale each) and back to values
  linear      products of two such operands, rows grouped by expert or dense
  gate_up     the same product for interleaved gate and up rows, with
              silu(gate) * up formed before anything is written
  decode      the expert FFN of 1 to 4 tokens over 4-bit experts, with the
              activations kept in fp32
  balance     the router's balance and z losses and per-expert counts
              (forward) and the gradient of the logits (backward)

With `own` false, run() computes them with elementary torch operations in 32
bits (64 for long sums); with `own` true it calls the framework.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32                                            # values that share a scale
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)       # magnitudes of the 3 low bits of a code


def listed():
    return [
        # one decode token's hidden state, and a prefill chunk of the model
        {"name": "quantize_token", "op": "quantize", "rows": 1, "cols": 2048, "dtype": "f32"},
        {"name": "quantize_chunk", "op": "quantize", "rows": 8192, "cols": 2048, "dtype": "bf16"},
        # the shared expert's down product over a chunk
        {"name": "linear_shared_chunk", "op": "linear", "tokens": 8192, "top_k": 0, "experts": 1,
         "cols": 768, "out": 2048, "dtype": "bf16"},
        # the routed experts' down products over a chunk: 81,920 rows in 512 groups
        {"name": "linear_experts_chunk", "op": "linear", "tokens": 8192, "top_k": 10, "experts": 512,
         "cols": 768, "out": 2048, "dtype": "f32"},
        # a small batch of prompts' last tokens through a small model's experts, ragged groups
        {"name": "linear_small_batch", "op": "linear", "tokens": 37, "top_k": 4, "experts": 60,
         "cols": 704, "out": 1040, "dtype": "f32"},
        # the routed experts' gate/up products: a chunk, and a batch of 64 sequences' next tokens
        {"name": "gate_up_chunk", "op": "gate_up", "tokens": 8192, "top_k": 10, "experts": 512,
         "cols": 2048, "out": 768, "dtype": "bf16"},
        {"name": "gate_up_batch", "op": "gate_up", "tokens": 64, "top_k": 10, "experts": 512,
         "cols": 2048, "out": 768, "dtype": "bf16"},
        # a decode step, and a verify step of one real and three drafted tokens
        {"name": "decode_token", "op": "decode", "tokens": 1, "top_k": 10, "experts": 128,
         "cols": 2048, "out": 768},
        {"name": "decode_verify", "op": "decode", "tokens": 4, "top_k": 10, "experts": 128,
         "cols": 2048, "out": 768},
        # one padded training batch of short sequences (padding masked) through a router
        {"name": "balance_short", "op": "balance", "back": False, "tokens": 131, "top_k": 6,
         "experts": 60, "seqs": 5, "masked": True},
        # a training step's packed sequences, forward and backward
        {"name": "balance_pack", "op": "balance", "back": False, "tokens": 65536, "top_k": 10,
         "experts": 512, "seqs": 16, "masked": False},
        {"name": "balance_pack_backward", "op": "balance", "back": True, "tokens": 65536, "top_k": 10,
         "experts": 512, "seqs": 16, "masked": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "gate_up", "decode", "balance"])
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 8192), "cols": BLOCK * _log(rng, 1, 64),
                "dtype": rng.choice(["f32", "bf16"])}
    if op in ("linear", "gate_up"):
        experts = rng.choice([1, _log(rng, 2, 512)])
        top_k = 0 if experts == 1 else rng.randint(1, min(10, experts))
        return {"op": op, "tokens": _log(rng, 1, 8192), "top_k": top_k, "experts": experts,
                "cols": BLOCK * rng.randint(1, 24 if op == "linear" else 64),
                "out": 16 * rng.randint(1, 128) if op == "linear" else BLOCK * rng.randint(1, 24),
                "dtype": rng.choice(["f32", "bf16"])}
    if op == "decode":
        experts = rng.randint(4, 128)
        return {"op": op, "tokens": rng.randint(1, 4), "top_k": rng.randint(1, min(10, experts)),
                "experts": experts, "cols": 64 * rng.randint(1, 32), "out": BLOCK * rng.randint(1, 24)}
    experts = rng.randint(2, 512)
    tokens = _log(rng, 1, 65536)
    return {"op": op, "back": rng.random() < 0.5, "tokens": tokens, "top_k": rng.randint(1, min(10, experts)),
            "experts": experts, "seqs": _log(rng, 1, min(64, tokens)), "masked": rng.random() < 0.5}


# --- microscaled 4-bit floats, plainly -----------------------------------------


def _plain_quantize(x):
    """Codes uint8 [..., cols / 2] (even value in the low nibble) and scales
    uint8 [..., cols / 32] (a power of two with bias 127): the scale is the
    block's largest magnitude's exponent less 2, values past 6 become 6,
    ties go to the code whose last bit is 0."""
    b = x.float().unflatten(-1, (-1, BLOCK))
    exp = torch.frexp(b.abs().amax(-1)).exponent.int() - 3
    exp = torch.where(b.abs().amax(-1) > 0, exp, -127).clamp(min=-127)
    a = b * ((127 - exp) << 23).view(torch.float32).unsqueeze(-1)
    m = a.abs()
    code = (m > 0.25).to(torch.uint8)
    for at, tie_up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (m >= at) if tie_up else (m > at)
    code += 8 * torch.signbit(a).to(torch.uint8)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (exp + 127).to(torch.uint8)


def _plain_values(codes, scales, dtype=torch.float32):
    lut = torch.tensor(GRID + tuple(-v for v in GRID), dtype=dtype, device=codes.device)
    pairs = torch.stack((lut.repeat(16), lut.repeat_interleave(16)), 1)     # both values of a byte
    v = pairs[codes.int()].flatten(-2).unflatten(-1, (-1, BLOCK))
    s = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=codes.device), scales.double() - 127)
    return (v * s.to(dtype).unsqueeze(-1)).flatten(-2)


# --- inputs --------------------------------------------------------------------


def _gen(case, seed):
    return torch.Generator(device="cuda").manual_seed(1000003 * (seed % (1 << 30)) + sum(map(ord, case["op"])))


def _hidden(g, rows, cols):
    """Hidden states: normal values, every 64th column eight times as large."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    x[:, ::64] *= 8
    return x


def _weights(g, mats, rows, cols):
    """Expert weights: normal, 1 / sqrt(cols) wide, quantized 16 matrices at a time."""
    codes = torch.empty((mats, rows, cols // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((mats, rows, cols // BLOCK), dtype=torch.uint8, device="cuda")
    for m in range(0, mats, 16):
        w = torch.randn((min(16, mats - m), rows, cols), generator=g, device="cuda") / math.sqrt(cols)
        codes[m:m + 16], scales[m:m + 16] = _plain_quantize(w)
    return codes, scales


def _logits(g, tokens, experts):
    """Router logits: normal, some experts more used than others."""
    return (torch.randn((tokens, experts), generator=g, device="cuda")
            + 0.5 * torch.randn((1, experts), generator=g, device="cuda"))


def prepare(case, seed):
    g = _gen(case, seed)
    s = dict(case)
    if case["op"] == "quantize":
        x = _hidden(g, case["rows"], case["cols"])
        s["x"] = x if case["dtype"] == "f32" else x.bfloat16()
        return s
    if case["op"] == "balance":
        T, E, k, S = case["tokens"], case["experts"], case["top_k"], case["seqs"]
        s["logits"] = _logits(g, T, E)
        s["idx"] = torch.topk(s["logits"], k).indices.int().contiguous()
        s["w"] = torch.softmax(torch.gather(s["logits"], 1, s["idx"].long()), 1)
        cuts = torch.randperm(max(T - 1, 1), generator=g, device="cuda")[:S - 1].sort().values + 1
        s["offsets"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)]).int()
        s["mask"] = ((torch.rand((T,), generator=g, device="cuda") < 0.8).to(torch.uint8)
                     if case["masked"] else None)
        if case["back"]:
            f = _plain_balance(s)
            s["counts"], s["n_tokens"] = f["counts"], f["n_tokens"]
            s["g_balance"] = 0.01 / S * (0.5 + torch.rand((S,), generator=g, device="cuda"))
            s["g_z"] = 0.001 / S * (0.5 + torch.rand((S,), generator=g, device="cuda"))
            s["dw"] = torch.randn((T, k), generator=g, device="cuda") / T
        return s
    T, E, k, K, N = (case[n] for n in ("tokens", "experts", "top_k", "cols", "out"))
    if case["op"] == "decode":
        lg = _logits(g, T, E)
        v, i = torch.topk(lg, k)
        s["slot"], s["w"] = i.int().contiguous(), torch.softmax(v, 1)
        s["x"] = torch.randn((T, K), generator=g, device="cuda")
        s["gate_up"] = _weights(g, E + 1, 2 * N, K)       # the last one is the shared expert
        s["down"] = _weights(g, E + 1, K, N)
        return s
    x = _hidden(g, T, K)
    if k == 0:                                            # every row, one matrix
        s["offsets"] = s["row_src"] = None
    else:
        i = torch.topk(_logits(g, T, E), k).indices
        order = torch.sort(i.flatten(), stable=True)
        s["row_src"] = order.indices.int()                # pair t * k + i of every row
        s["offsets"] = torch.searchsorted(order.values, torch.arange(E + 1, device="cuda")).int()
        if case["op"] == "linear":                        # rows already in group order, as gate_up leaves them
            x = _hidden(g, T * k, K)
            s["row_src"] = None
        s["most"] = int(s["offsets"].diff().max())
    s["a"] = _plain_quantize(x)
    s["b"] = _weights(g, E, N if case["op"] == "linear" else 2 * N, K)
    return s


# --- the operators, plainly ----------------------------------------------------


def _rounded(v, case):
    return v.to(torch.float32 if case["dtype"] == "f32" else torch.bfloat16)


def _plain_product(s):
    """fp32 [rows, out]: each row of `a` times its group's matrix, the groups
    padded to the longest and multiplied as one batch."""
    a, b = _plain_values(*s["a"]), _plain_values(*s["b"])
    if s["offsets"] is None:
        return a @ b[0].t()
    off = s["offsets"].long()
    if s["row_src"] is not None:
        a = a[s["row_src"].long() // s["top_k"]]
    at = off[:-1, None] + torch.arange(s["most"], device=off.device)       # row of every place of the batch
    inside = at < off[1:, None]
    cols = a[at.clamp(max=a.shape[0] - 1)].transpose(1, 2).contiguous()
    return torch.bmm(b, cols).transpose(1, 2)[inside]                      # groups ascending: the rows in order


def _plain_ffn(x, gu, dn):
    """x [n, d], gu [n, 2f, d], dn [n, d, f]: the expert FFN of each row."""
    h = torch.matmul(gu, x.unsqueeze(-1)).squeeze(-1)
    h = h[:, 0::2] * torch.sigmoid(h[:, 0::2]) * h[:, 1::2]
    return torch.matmul(dn, h.unsqueeze(-1)).squeeze(-1)


def _plain_decode(s, dtype=torch.float32):
    T, k = s["slot"].shape
    at = torch.cat([s["slot"].long(), torch.full((T, 1), s["experts"], device="cuda")], 1).flatten()
    gu = _plain_values(s["gate_up"][0][at], s["gate_up"][1][at], dtype)
    dn = _plain_values(s["down"][0][at], s["down"][1][at], dtype)
    x = s["x"].to(dtype)
    y = _plain_ffn(x.repeat_interleave(k + 1, 0), gu, dn).unflatten(0, (T, k + 1))
    w = torch.cat([s["w"].to(dtype), torch.ones((T, 1), dtype=dtype, device="cuda")], 1)
    return x + (y * w.unsqueeze(-1)).sum(1)


def _rows_of(s):
    """(sequence of every row, whether it takes part)."""
    T = s["logits"].shape[0]
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["offsets"], t, right=True).long() - 1
    part = (seq >= 0) & (seq < s["seqs"])
    if s["mask"] is not None:
        part &= s["mask"] != 0
    return seq.clamp(0, s["seqs"] - 1), part


def _plain_balance(s):
    E, k, S = s["experts"], s["top_k"], s["seqs"]
    seq, part = _rows_of(s)
    lse = torch.logsumexp(s["logits"], 1)
    rows = ((torch.arange(S, device="cuda")[:, None] == seq) & part).double()         # [S, T]: the rows of each
    P = rows @ torch.softmax(s["logits"], 1).double()
    z = rows @ (lse.double() ** 2)
    n = rows.sum(1).int()
    at = torch.where(part, seq, S)[:, None] * E + s["idx"]
    c = torch.bincount(at.flatten(), minlength=(S + 1) * E)[:S * E].view(S, E).int()
    m = n.double().clamp(min=1)
    return {"balance": (E / (k * m * m) * (c * P).sum(1)).float(), "z": (z / m).float(), "counts": c,
            "prob_sum": P.float(), "n_tokens": n}


def _plain_balance_backward(s, dtype=torch.float32):
    E, k = s["experts"], s["top_k"]
    seq, part = _rows_of(s)
    l = s["logits"].to(dtype)
    p, lse = torch.softmax(l, 1), torch.logsumexp(l, 1, keepdim=True)
    n = s["n_tokens"].to(dtype).clamp(min=1)
    c = s["counts"] - (s["counts"].sum(1, keepdim=True) // E)              # the mean off: p sums to 1
    c = c.to(dtype)[seq]
    d = (s["g_balance"].to(dtype) * E / (k * n * n))[seq, None] * p * (c - (c * p).sum(1, keepdim=True))
    d += (s["g_z"].to(dtype) * 2 / n)[seq, None] * lse * p
    w, dw = s["w"].to(dtype), s["dw"].to(dtype)
    d.scatter_add_(1, s["idx"].long(), w * (dw - (w * dw).sum(1, keepdim=True)))
    return d * part[:, None]


def run(s):
    op = s["op"]
    if own:
        import bit_expert_ffn_top_amd as bf
        if op == "quantize":
            return bf.mxfp4_dequantize(bf.mxfp4_quantize(s["x"]), dtype=torch.bfloat16)
        if op == "decode":
            return bf.mxfp4_ffn_decode(bf.Mxfp4(*s["gate_up"]), bf.Mxfp4(*s["down"]), s["x"], s["slot"], s["w"],
                                       shared_slot=s["experts"])
        if op == "balance":
            if s["back"]:
                return bf.route_backward(s["logits"], s["idx"], s["counts"], s["n_tokens"],
                                         g_balance=s["g_balance"], g_z=s["g_z"], w=s["w"], dw=s["dw"],
                                         seq_offsets=s["offsets"], mask=s["mask"])
            return bf.route_balance(s["logits"], s["idx"], seq_offsets=s["offsets"], mask=s["mask"])._asdict()
        out = torch.float32 if s["dtype"] == "f32" else torch.bfloat16
        call = bf.mxfp4_linear if op == "linear" else bf.mxfp4_gate_up
        return call(bf.Mxfp4(*s["a"]), bf.Mxfp4(*s["b"]), offsets=s["offsets"], row_src=s["row_src"],
                    src_div=max(s["top_k"], 1), dtype=out)
    if op == "quantize":
        return _plain_values(*_plain_quantize(s["x"])).bfloat16()
    if op == "decode":
        return _plain_decode(s)
    if op == "balance":
        return _plain_balance_backward(s) if s["back"] else _plain_balance(s)
    y = _plain_product(s)
    if op == "gate_up":
        y = y[:, 0::2] * torch.sigmoid(y[:, 0::2]) * y[:, 1::2]
    return _rounded(y, s)


def work(case):
    """Each input once, each output once; of the expert matrices those that are used."""
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * ((4 if case["dtype"] == "f32" else 2) + 2), "flops": 4 * n}
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    if op == "balance":
        n = T * E
        per_token = 4 * k + (1 if case["masked"] else 0)
        if case["back"]:
            return {"bytes": 8 * n + T * (per_token + 8 * k) + 4 * E * case["seqs"], "flops": 12 * n}
        return {"bytes": 4 * n + T * per_token + 8 * E * case["seqs"], "flops": 6 * n}
    K, N = case["cols"], case["out"]
    row = K / 2 + K / BLOCK
    if op == "decode":
        used = E * (1 - (1 - 1 / E) ** (T * k)) + 1       # expected distinct experts, and the shared one
        used = min(used, T * k + 1)
        return {"bytes": used * (2 * N * row + K * (N / 2 + N / BLOCK)) + 8 * T * K + 8 * T * k,
                "flops": 6 * T * (k + 1) * N * K}
    rows = T * max(k, 1)
    used = min(E * (1 - (1 - 1 / E) ** rows), rows) if E > 1 else 1
    n_out = N if op == "linear" else 2 * N
    a_rows = T if op == "gate_up" else rows
    return {"bytes": used * n_out * row + a_rows * row + rows * N * (4 if case["dtype"] == "f32" else 2),
            "flops": 2 * rows * n_out * K}


# --- the definitions in 64 bits, apart from the plain forms --------------------


def _exact_grid(x):
    """x float64 [..., 32] on the grid of its block: the nearest multiple of
    the spacing at each magnitude, ties to the even multiple."""
    top = np.abs(x).max(-1, keepdims=True)
    e = np.floor(np.log2(np.where(top > 0, top, 1.0)))
    e = np.where(np.ldexp(1.0, e.astype(int)) > top, e - 1, e)
    e = np.where(top > 0, np.maximum(e - 2, -127), -127).astype(int)
    m = np.abs(x) / np.ldexp(1.0, e)
    step = np.where(m < 2, 0.5, np.where(m < 4, 1.0, 2.0))
    return np.copysign(np.minimum(np.round(m / step) * step, 6.0) * np.ldexp(1.0, e), x)


def _exact_values(codes, scales):
    """float64 values, from the fields of each code."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()
    e, m = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * (1 << (e - 1).clamp(min=0)).double())
    v = torch.where(c >= 8, -v, v).unflatten(-1, (-1, BLOCK))
    return torch.ldexp(v, (scales.int() - 127).unsqueeze(-1)).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = s["x"].double().cpu().numpy()
        return torch.from_numpy(_exact_grid(x.reshape(x.shape[0], -1, BLOCK)).reshape(x.shape))
    if op == "decode":
        rows = []
        for t in range(case["tokens"]):
            y = s["x"][t].double()
            terms = [(int(e), float(w)) for e, w in zip(s["slot"][t].tolist(), s["w"][t].tolist())]
            for e, w in terms + [(case["experts"], 1.0)]:
                h = _exact_values(*(v[e] for v in s["gate_up"])) @ s["x"][t].double()
                g, u = h[0::2], h[1::2]
                y = y + w * (_exact_values(*(v[e] for v in s["down"])) @ (g / (1 + torch.exp(-g)) * u))
            rows.append(y)
        return torch.stack(rows)
    if op == "balance":
        return _exact_balance(s)
    a = _exact_values(*s["a"])
    off = [0, a.shape[0]] if s["offsets"] is None else s["offsets"].tolist()
    src = None if s["row_src"] is None else s["row_src"].long() // case["top_k"]
    parts = []
    for e in range(len(off) - 1):
        if off[e] == off[e + 1]:
            continue
        rows = a[off[e]:off[e + 1]] if src is None else a[src[off[e]:off[e + 1]]]
        parts.append(rows @ _exact_values(s["b"][0][e], s["b"][1][e]).t().contiguous())
    y = torch.cat(parts)
    if op == "gate_up":
        y = y[:, 0::2] / (1 + torch.exp(-y[:, 0::2])) * y[:, 1::2]
    return y


def _exact_balance(s):
    """The losses and, for the backward pass, their gradient, sequence by
    sequence: balance = E / (k n^2) sum_e count_e sum_t p_te, z = mean lse^2."""
    E, k, S = s["experts"], s["top_k"], s["seqs"]
    off = s["offsets"].tolist()
    l = s["logits"].double()
    out = {n: [] for n in ("balance", "z", "counts", "prob_sum", "n_tokens")}
    grad = torch.zeros_like(l)
    for q in range(S):
        rows = torch.arange(off[q], off[q + 1], device="cuda")
        if s["mask"] is not None:
            rows = rows[s["mask"][rows].bool()]
        x = l[rows]
        top = x.amax(1, keepdim=True) if rows.numel() else x[:, :1]
        ex = torch.exp(x - top)
        lse = top + torch.log(ex.sum(1, keepdim=True))
        p = ex / ex.sum(1, keepdim=True)
        n = max(rows.numel(), 1)
        c = torch.bincount(s["idx"][rows].flatten().long(), minlength=E)
        out["counts"].append(c)
        out["prob_sum"].append(p.sum(0))
        out["n_tokens"].append(rows.numel())
        out["balance"].append((c.double() @ p.sum(0)) * E / (k * n * n))
        out["z"].append((lse ** 2).sum() / n)
        if s["back"]:
            f = c.double()
            d = s["g_balance"][q].double() * E / (k * n * n) * p * (f - (p @ f)[:, None])
            d = d + s["g_z"][q].double() * 2 / n * lse * p
            w, dw = s["w"][rows].double(), s["dw"][rows].double()
            hot = torch.nn.functional.one_hot(s["idx"][rows].long(), E).double()
            grad[rows] = d + ((w * (dw - (w * dw).sum(1, keepdim=True)))[:, :, None] * hot).sum(1)
    if s["back"]:
        return grad
    return {"balance": torch.stack(out["balance"]), "z": torch.stack(out["z"]), "counts": None,
            "prob_sum": torch.stack(out["prob_sum"]), "n_tokens": None}
