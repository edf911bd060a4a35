"""More operators measured in this repository, with their plain forms.

What a step for many requests needs around the routed experts:

  dispatch   tokens sorted by expert: the pairs' groups and their rows
             (forward), and the gradient of the tokens (backward)
  combine    the experts' rows back in the tokens' order, with the routing
             weights applied (forward), and the gradients of the rows and of
             the weights (backward)
  lora       low-rank adapters of many requests beside a shared projection
  verify     drafted tokens accepted or replaced, by the target's and the
             drafts' probabilities and given random numbers

With `own` false, run() computes them with elementary torch operations in 32
bits (64 for what lies next to a border); with `own` true it calls the framework.
"""
import math

import torch

own = False


def listed():
    return [
        # the next tokens of 64 sequences to their experts, and a prefill chunk
        {"name": "dispatch_batch", "op": "dispatch", "back": False, "tokens": 64, "top_k": 10,
         "experts": 512, "cols": 2048, "dtype": "bf16", "padded": False},
        {"name": "dispatch_chunk", "op": "dispatch", "back": False, "tokens": 8192, "top_k": 10,
         "experts": 512, "cols": 2048, "dtype": "bf16", "padded": False},
        # the tokens' gradient in a training step over a chunk
        {"name": "dispatch_chunk_backward", "op": "dispatch", "back": True, "tokens": 8192, "top_k": 10,
         "experts": 512, "cols": 2048, "dtype": "bf16", "padded": False},
        # a verify step of one real and three drafted tokens; a chunk; a training
        # step over a chunk; and a small model's padded batch in fp32, odd sizes
        {"name": "combine_verify", "op": "combine", "back": False, "tokens": 4, "top_k": 10,
         "experts": 512, "cols": 2048, "dtype": "f32", "padded": False},
        {"name": "combine_chunk", "op": "combine", "back": False, "tokens": 8192, "top_k": 10,
         "experts": 512, "cols": 2048, "dtype": "bf16", "padded": False},
        {"name": "combine_chunk_backward", "op": "combine", "back": True, "tokens": 8192, "top_k": 10,
         "experts": 512, "cols": 2048, "dtype": "bf16", "padded": False},
        {"name": "combine_small_backward", "op": "combine", "back": True, "tokens": 1037, "top_k": 6,
         "experts": 60, "cols": 1044, "dtype": "f32", "padded": True},
        # a single token, the next tokens of 64 sequences with one adapter each out
        # of 48, and a chunk of eight ragged prompts
        {"name": "lora_token", "op": "lora", "tokens": 1, "seqs": 1, "adapters": 16, "rank": 16,
         "cols": 2048, "out": 1536, "dtype": "f32"},
        {"name": "lora_batch", "op": "lora", "tokens": 64, "seqs": 64, "adapters": 48, "rank": 16,
         "cols": 2048, "out": 1536, "dtype": "bf16"},
        {"name": "lora_prompts", "op": "lora", "tokens": 8192, "seqs": 8, "adapters": 48, "rank": 64,
         "cols": 2048, "out": 2048, "dtype": "bf16"},
        # three drafts of one sequence, and of 64 sequences at once with fewer
        # drafts for some of them
        {"name": "verify_one", "op": "verify", "seqs": 1, "drafts": 3, "vocab": 131072, "from_model": True,
         "ragged": False},
        {"name": "verify_batch", "op": "verify", "seqs": 64, "drafts": 3, "vocab": 131072, "from_model": True,
         "ragged": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dispatch", "combine", "lora", "verify"])
    dtype = rng.choice(["f32", "bf16"])
    tokens = _log(rng, 1, 8192 if dtype == "bf16" else 4096)
    if op in ("dispatch", "combine"):
        experts = rng.randint(2, 512)
        return {"op": op, "back": rng.random() < 0.5, "tokens": tokens, "top_k": rng.randint(1, min(10, experts)),
                "experts": experts, "cols": 4 * _log(rng, 16, 512), "dtype": dtype, "padded": rng.random() < 0.3}
    if op == "lora":
        seqs = tokens if rng.random() < 0.3 and tokens <= 512 else _log(rng, 1, min(256, tokens))
        return {"op": op, "tokens": tokens, "seqs": seqs, "adapters": _log(rng, 1, 64),
                "rank": 8 * rng.randint(1, 8), "cols": 32 * rng.randint(2, 64), "out": 16 * rng.randint(2, 128),
                "dtype": dtype}
    drafts = rng.randint(1, 7)
    return {"op": op, "seqs": _log(rng, 1, 256 // (drafts + 1)), "drafts": drafts,
            "vocab": _log(rng, 1000, 131072), "from_model": rng.random() < 0.7, "ragged": rng.random() < 0.5}


# --- inputs --------------------------------------------------------------------


def _gen(case, seed):
    return torch.Generator(device="cuda").manual_seed(1000003 * (seed % (1 << 30)) + sum(map(ord, case["op"])))


def _type(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _normal(g, case, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(_type(case))


def _routing(g, case):
    """(chosen experts int32 [T, k], weights): some experts more used than
    others; in a padded batch about a tenth of the tokens choose none."""
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    logits = (torch.randn((T, E), generator=g, device="cuda")
              + 0.5 * torch.randn((1, E), generator=g, device="cuda"))
    v, i = torch.topk(logits, k)
    if case["padded"]:
        i[torch.rand((T,), generator=g, device="cuda") < 0.1] = -1
    return i.int().contiguous(), torch.softmax(v, 1)


def prepare(case, seed):
    g = _gen(case, seed)
    s = dict(case)
    if case["op"] in ("dispatch", "combine"):
        T, k, d = case["tokens"], case["top_k"], case["cols"]
        s["idx"], s["w"] = _routing(g, case)
        if case["op"] == "dispatch" and not case["back"]:
            s["x"] = _normal(g, case, T, d)
            s["out"] = torch.zeros((T * k, d), dtype=_type(case), device="cuda")
            return s
        s["pair_pos"] = _plain_groups(s)["pair_pos"]      # as the step's dispatch left it
        s["rows"] = _normal(g, case, T * k, d)
        if case["op"] == "combine" and case["back"]:
            s["dy"] = _normal(g, case, T, d)
            s["out"] = torch.zeros((T * k, d), dtype=_type(case), device="cuda")
        elif case["op"] == "combine":
            s["base"] = _normal(g, case, T, d)            # residual or shared expert
        return s
    if case["op"] == "lora":
        T, S, n, r, K, N = (case[v] for v in ("tokens", "seqs", "adapters", "rank", "cols", "out"))
        s["x"], s["base"] = _normal(g, case, T, K), _normal(g, case, T, N)
        s["a"] = (torch.randn((n, r, K), generator=g, device="cuda") / math.sqrt(K)).bfloat16()
        s["b"] = (torch.randn((n, N, r), generator=g, device="cuda") / math.sqrt(r)).bfloat16()
        s["scale"] = 0.25 + torch.rand((n,), generator=g, device="cuda")
        s["adapter"] = torch.randint(0, n, (S,), generator=g, device="cuda").int()
        if S > 4:                                         # some requests go without one
            s["adapter"][torch.rand((S,), generator=g, device="cuda") < 0.1] = -1
        s["offsets"] = None                               # a row for every request
        s["most"] = 1
        if S != T:
            cuts = torch.randperm(T - 1, generator=g, device="cuda")[:S - 1].sort().values + 1
            s["offsets"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)]).int()
            s["most"] = int(s["offsets"].diff().max())
        return s
    B, n, V = case["seqs"], case["drafts"], case["vocab"]
    logits = 3 * torch.randn((B, n + 1, V), generator=g, device="cuda")
    s["p"] = torch.softmax(logits, -1)
    s["q"] = None
    near = torch.softmax(logits[:, :n] + 0.5 * torch.randn((B, n, V), generator=g, device="cuda"), -1)
    s["draft"] = torch.multinomial(near.flatten(0, 1), 1, generator=g).view(B, n).int()
    if case["from_model"]:
        s["q"] = near
    s["u_accept"] = torch.rand((B, n), generator=g, device="cuda")
    s["u_sample"] = torch.rand((B,), generator=g, device="cuda")
    s["n_draft"] = (torch.randint(0, n + 1, (B,), generator=g, device="cuda").int() if case["ragged"] else None)
    return s


# --- the operators, plainly ----------------------------------------------------


def _plain_groups(s):
    """Rows of the pairs, groups ascending by expert, in t, then i order inside."""
    T, k = s["idx"].shape
    E = s["experts"]
    e = s["idx"].flatten()
    e = torch.where((e >= 0) & (e < E), e, E)
    order = torch.sort(e, stable=True)
    offsets = torch.searchsorted(order.values, torch.arange(E + 1, device="cuda", dtype=torch.int32)).int()
    at = torch.arange(T * k, device="cuda", dtype=torch.int32)
    pos = torch.empty_like(at)
    pos[order.indices] = torch.where(order.values < E, at, -1)
    return {"offsets": offsets, "pair_pos": pos.view(T, k), "token": order.indices // k, "grouped": at < offsets[E]}


def _plain_dispatch(s):
    f = _plain_groups(s)
    rows = torch.where(f["grouped"][:, None], s["x"][f["token"]], 0)
    return {"rows": rows, "offsets": f["offsets"], "pair_pos": f["pair_pos"]}


def _rows_of_tokens(s):
    """fp32 [T, k, d]: the row of every pair, zeros where it has none."""
    pos = s["pair_pos"].long()
    return s["rows"].float()[pos.clamp(min=0)] * (pos >= 0)[..., None]


def _plain_combine(s, weights, base):
    y = _rows_of_tokens(s)
    if weights:
        y = y * s["w"][..., None]
    y = y.sum(1)
    if base:
        y = s["base"].float() + y
    return y.to(_type(s))


def _plain_combine_backward(s):
    pos = s["pair_pos"].long()
    dy = s["dy"].float()
    dw = (_rows_of_tokens(s) * dy[:, None]).sum(-1)
    grad = (s["w"][..., None] * dy[:, None]).to(_type(s))
    drows = torch.zeros_like(s["rows"])
    drows[pos[pos >= 0]] = grad[pos >= 0]
    return {"drows": drows, "dw": dw}


def _plain_lora(s):
    """The requests' rows padded to the longest request, as batches."""
    n, T = s["adapters"], s["tokens"]
    off = s["offsets"]
    if off is None:
        off = torch.arange(T + 1, device="cuda", dtype=torch.int32)
    at = off[:-1, None].long() + torch.arange(s["most"], device="cuda")
    inside = at < off[1:, None]
    who = s["adapter"].long()
    has = (who >= 0) & (who < n)
    who = who.clamp(0, n - 1)
    x = s["x"].float()[at.clamp(max=T - 1)]
    h = torch.bmm(x, s["a"].float()[who].transpose(1, 2).contiguous())
    h = h * (s["scale"][who] * has)[:, None, None]
    delta = torch.bmm(h, s["b"].float()[who].transpose(1, 2).contiguous())
    return (s["base"].float() + delta[inside]).to(_type(s))


def _plain_verify(s):
    B, n = s["draft"].shape
    p, q, x = s["p"], s["q"], s["draft"].long()
    b, i = torch.arange(B, device="cuda"), torch.arange(n, device="cuda")
    given = torch.full((B,), n, device="cuda") if s["n_draft"] is None else s["n_draft"].long()
    px = p[b[:, None], i, x].double()
    qx = torch.ones_like(px) if q is None else q[b[:, None], i, x].double()
    ok = (s["u_accept"].double() * qx < px) & (i < given[:, None])
    m = ok.long().cumprod(1).sum(1)                       # drafts accepted
    row = p[b, m].double()
    at = m.clamp(max=n - 1)
    if q is None:
        less = torch.zeros_like(row)
        less[b, x[b, at]] = row[b, x[b, at]]
    else:
        less = q[b, at].double()
    rest = (row - less * (m < given)[:, None]).clamp(min=0)
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, row)
    cum = rest.cumsum(1)
    pick = (cum <= (s["u_sample"].double() * cum[:, -1])[:, None]).sum(1)
    last = torch.where(rest > 0, torch.arange(rest.shape[1], device="cuda"), -1).amax(1)
    pick = torch.minimum(pick, last)
    place = torch.arange(n + 1, device="cuda")
    tokens = torch.cat([x, x[:, :1]], 1)
    tokens = torch.where(place < m[:, None], tokens, torch.where(place == m[:, None], pick[:, None], -1))
    return {"tokens": tokens.int(), "n_accepted": m.int()}


def run(s):
    op = s["op"]
    if own:
        import bit_expert_ffn_top_amd as bf
        if op == "dispatch":
            if s["back"]:
                return bf.dispatch_backward(s["rows"], s["pair_pos"])
            return bf.dispatch(s["x"], s["idx"], s["experts"], rows=s["out"])._asdict()
        if op == "combine":
            if s["back"]:
                drows, dw = bf.combine_backward(s["dy"], s["rows"], s["pair_pos"], s["w"], drows=s["out"])
                return {"drows": drows, "dw": dw}
            return bf.combine_rows(s["rows"], s["pair_pos"], s["w"], base=s["base"])
        if op == "lora":
            return bf.lora(s["base"], s["x"], s["a"], s["b"], s["adapter"], seq_offsets=s["offsets"],
                           scale=s["scale"])
        tokens, n_accepted = bf.verify_drafts(s["p"], s["q"], s["draft"], s["u_accept"], s["u_sample"],
                                              n_draft=s["n_draft"])
        return {"tokens": tokens, "n_accepted": n_accepted}
    if op == "dispatch":
        return _plain_combine(s, False, False) if s["back"] else _plain_dispatch(s)
    if op == "combine":
        return _plain_combine_backward(s) if s["back"] else _plain_combine(s, True, True)
    if op == "lora":
        return _plain_lora(s)
    return _plain_verify(s)


def work(case):
    """Each input once, each output once; of the adapters those that are used, of
    the probabilities the rows that are sampled from and the drafts' own."""
    op = case["op"]
    if op == "verify":
        B, n, V = case["seqs"], case["drafts"], case["vocab"]
        per = 8 if case["from_model"] else 4
        return {"bytes": B * (V * per + n * (4 + 4 + per) + 4 * (n + 2)), "flops": 3 * B * V}
    e = 4 if case["dtype"] == "f32" else 2
    T = case["tokens"]
    if op == "lora":
        S, n, r, K, N = (case[v] for v in ("seqs", "adapters", "rank", "cols", "out"))
        used = min(n * (1 - (1 - 1 / n) ** S), S) if n > 1 else 1
        return {"bytes": T * (K + 2 * N) * e + used * 2 * r * (K + N) + 8 * S, "flops": 2 * T * r * (K + N)}
    k, d = case["top_k"], case["cols"]
    token, pairs = T * d * e, T * k * d * e               # bytes of the tokens' and of the pairs' rows
    if op == "dispatch":
        if case["back"]:
            return {"bytes": pairs + token + 4 * T * k, "flops": T * k * d}
        return {"bytes": pairs + token + 8 * T * k, "flops": T * k}
    if case["back"]:
        return {"bytes": 2 * pairs + token + 12 * T * k, "flops": 3 * T * k * d}
    return {"bytes": pairs + 2 * token + 8 * T * k, "flops": 2 * T * k * d}


# --- the definitions in 64 bits, apart from the plain forms --------------------


def _exact_positions(idx, experts):
    """Row of every pair, counted expert by expert; -1 for ids of no expert."""
    e = idx.flatten().long().cpu()
    pos = torch.full_like(e, -1)
    at = 0
    for x in range(experts):
        mine = (e == x).nonzero().flatten()
        pos[mine] = torch.arange(at, at + mine.numel())
        at += mine.numel()
    return pos.view(idx.shape).to(idx.device)


def exact(case, seed):
    if case["op"] == "verify":
        return None                                       # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "lora":
        y = s["base"].double()
        off = list(range(case["tokens"] + 1)) if s["offsets"] is None else s["offsets"].tolist()
        for q, who in enumerate(s["adapter"].tolist()):
            if 0 <= who < case["adapters"]:
                x = s["x"][off[q]:off[q + 1]].double()
                h = x @ s["a"][who].double().t().contiguous()
                y[off[q]:off[q + 1]] += float(s["scale"][who]) * (h @ s["b"][who].double().t().contiguous())
        return y
    T, k, d = case["tokens"], case["top_k"], case["cols"]
    pos = _exact_positions(s["idx"], case["experts"])
    if case["op"] == "dispatch" and not case["back"]:
        rows = torch.zeros((T * k, d), dtype=torch.float64, device="cuda")
        for i in range(k):
            there = (pos[:, i] >= 0).nonzero().flatten()
            rows[pos[there, i]] = s["x"][there].double()
        return {"rows": rows, "offsets": None, "pair_pos": None}
    if case["op"] == "combine" and case["back"]:
        drows = torch.zeros((T * k, d), dtype=torch.float64, device="cuda")
        dw = torch.zeros((T, k), dtype=torch.float64, device="cuda")
        for i in range(k):
            there = (pos[:, i] >= 0).nonzero().flatten()
            p, dy = pos[there, i], s["dy"][there].double()
            drows[p] = s["w"][there, i].double()[:, None] * dy
            dw[there, i] = (dy * s["rows"][p].double()).sum(1)
        return {"drows": drows, "dw": dw}
    y = s["base"].double() if case["op"] == "combine" else torch.zeros((T, d), dtype=torch.float64, device="cuda")
    for i in range(k):
        there = (pos[:, i] >= 0).nonzero().flatten()
        term = s["rows"][pos[there, i]].double()
        y[there] += term * s["w"][there, i].double()[:, None] if case["op"] == "combine" else term
    return y
