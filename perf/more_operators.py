"""The operators around a layer's 4-bit products, cache and attention, measured:
their cases, their plain forms in elementary torch operations (FP32, FP64 where
FP32 loses what matters, rounded once at the end) and the calls a user makes of
them.

  rotary   rotary positions of queries and keys, between the fused projection
           and the cache: pairs (x[i], x[i + r/2]) or (x[2i], x[2i + 1]) of the
           first r elements of every head turned by position * frequency[i]
  route    scores of experts, softmax or sigmoid, a bias that only chooses,
           groups of which some are open, the k best and their weights
  rows     a token's row to its experts' places, in the order that the experts'
           products take (row offsets per expert), and the weighted sum back
  prompt   causal attention of packed sequences in BF16, each sequence's
           queries being the last of its keys (a chunk behind a context that
           was read back from the cache, or a whole prompt)
"""
import math

import torch

own = False

DEVICE = "cuda"


# ---- cases -----------------------------------------------------------------

def _rotary(name, tokens, heads, kv_heads, head_dim, dims, interleaved=False, dtype="bf16", start=0,
            base=10000.0, factor=1.0, method="none", inverse=False):
    return {"name": name, "op": "rotary", "tokens": tokens, "heads": heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "dims": dims, "interleaved": interleaved, "dtype": dtype, "start": start,
            "base": base, "factor": factor, "method": method, "inverse": inverse}


def _route(name, tokens, experts, top_k, scoring, dtype="f32", bias=False, groups=1, top_groups=1,
           renormalize=True, scale=1.0):
    return {"name": name, "op": "route", "tokens": tokens, "experts": experts, "top_k": top_k,
            "scoring": scoring, "dtype": dtype, "bias": bias, "groups": groups, "top_groups": top_groups,
            "renormalize": renormalize, "scale": scale}


def _rows(name, tokens, experts, top_k, hidden, dtype="bf16", add=True):
    return {"name": name, "op": "rows", "tokens": tokens, "experts": experts, "top_k": top_k,
            "hidden": hidden, "dtype": dtype, "add": add}


def _prompt(name, batch, short, long, heads, kv_heads, head_dim, cached=0):
    return {"name": name, "op": "prompt", "batch": batch, "short": short, "long": long, "heads": heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "cached": cached}


def listed():
    return [
        # a decode step's new tokens of 64 samples, 64 heads on 8: latency
        _rotary("rotary_decode_64", 64, 64, 8, 128, 128, start=4000),
        # packed prompts far into a context that was stretched sixteenfold
        _rotary("rotary_prompt_8192", 8192, 32, 8, 128, 128, interleaved=True, start=90000, factor=16.0,
                method="parts"),
        # a third of each wide head, FP32 from the projection, turned back, an odd number of tokens
        _rotary("rotary_odd_777", 777, 5, 1, 192, 64, dtype="f32", start=1000000, factor=4.0,
                method="positions", inverse=True),
        # a decode batch: 8 of 256 experts from four of eight groups, balanced by a bias
        _route("route_64x256", 64, 256, 8, "sigmoid", bias=True, groups=8, top_groups=4, scale=2.5),
        # a prefill's tokens over 128 experts, scores of a BF16 projection (with ties)
        _route("route_8192x128", 8192, 128, 8, "softmax", dtype="bf16"),
        # a decode batch's rows to 8 of 32 experts each and back
        _rows("rows_64x7168", 64, 32, 8, 7168),
        # a prefill's rows to 8 of 128 experts each and back
        _rows("rows_8192x2048", 8192, 128, 8, 2048),
        # one prompt of a few hundred tokens: latency
        _prompt("prompt_1x512", 1, 512, 512, 32, 8, 128),
        # prompts of mixed length packed into one call
        _prompt("prompt_16x2048", 16, 33, 2048, 32, 8, 128),
        # one long prompt: the largest
        _prompt("prompt_1x8192", 1, 8192, 8192, 32, 8, 128),
        # chunks of 512 tokens behind contexts read back from the cache
        _prompt("prompt_chunk_4x512", 4, 512, 512, 32, 8, 128, cached=6001),
        # odd lengths from nothing up, few heads of 64
        _prompt("prompt_odd_13x300", 13, 0, 300, 12, 3, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotary", "route", "rows", "prompt", "prompt", "prompt"))
    if op == "rotary":
        head_dim = rng.choice((64, 80, 96, 128, 128, 192, 256))
        dims = head_dim if rng.random() < 0.6 else 2 * rng.randint(4, head_dim // 2)
        method = rng.choice(("none", "positions", "base", "parts"))
        kv_heads = rng.randint(0, 8)
        return _rotary("", _log(rng, 1, 8192), max(1, kv_heads) * rng.randint(1, 8), kv_heads, head_dim, dims,
                       rng.random() < 0.5, rng.choice(("bf16", "bf16", "f32")), _log(rng, 1, 1000000),
                       rng.choice((10000.0, 500000.0)), 1.0 if method == "none" else float(rng.randint(2, 32)),
                       method, rng.random() < 0.3)
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        experts = groups * rng.randint(4, max(4, 512 // groups))
        top_groups = rng.randint(1, groups)
        return _route("", _log(rng, 1, 16384), experts, rng.randint(1, min(8, top_groups * (experts // groups))),
                      rng.choice(("softmax", "sigmoid")), rng.choice(("bf16", "f32")), rng.random() < 0.5, groups,
                      top_groups, rng.random() < 0.7, rng.choice((1.0, 2.5)))
    if op == "rows":
        experts, hidden = rng.randint(2, 256), _log(rng, 64, 7168)
        top_k = rng.randint(1, min(8, experts))
        return _rows("", _log(rng, 1, max(2, min(16384, (1 << 27) // (top_k * hidden)))), experts, top_k, hidden,
                     rng.choice(("bf16", "bf16", "f32")), rng.random() < 0.5)
    kv_heads = rng.randint(1, 8)
    heads = kv_heads * rng.choice((1, 2, 4, 5, 8))
    head_dim = rng.choice((64, 128, 128, 128, 192, 256))
    batch, long = _log(rng, 1, 32), _log(rng, 16, 8192)
    cached = rng.choice((0, 0, _log(rng, 16, 8192)))
    case = _prompt("", batch, rng.randint(0, long), long, heads, kv_heads, head_dim, cached)
    # fewer sequences, then shorter ones, until their work is at most a third of the largest's
    while work(case)["flops"] > 1.8e11:
        if case["batch"] > 1:
            case["batch"] //= 2
        else:
            case["long"] = case["long"] * 2 // 3
            case["short"] = min(case["short"], case["long"])
    return case


# ---- inputs ----------------------------------------------------------------

def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _projected(gen, tokens, heads, head_dim):
    """Heads as a fused projection leaves them: per-token gains and a few strong channels."""
    x = torch.randn((tokens, heads, head_dim), generator=gen, device=DEVICE)
    x *= torch.exp(0.3 * torch.randn((tokens, 1, 1), generator=gen, device=DEVICE))
    x[..., torch.randperm(head_dim, generator=gen, device=DEVICE)[:max(1, head_dim // 32)]] *= 3.0
    return x


def _prepare_rotary(case, gen):
    tokens, heads, kv_heads, d = (case[n] for n in ("tokens", "heads", "kv_heads", "head_dim"))
    # queries and keys lie in the projection's rows, the values behind them
    qkv = _projected(gen, tokens, heads + 2 * kv_heads, d).to(_dtype(case))
    # a few sequences packed one behind the other, each from its own position on
    parts = 1 + tokens // 1500
    first = torch.randint(0, 1 + case["start"] // 8, (parts,), generator=gen, device=DEVICE)
    at = torch.arange(tokens, device=DEVICE)
    positions = case["start"] + first[at * parts // tokens] + at % -(-tokens // parts)
    frequencies, amplitude = _frequencies(case)
    return {"case": case, "q": qkv[:, :heads], "k": qkv[:, heads:heads + kv_heads] if kv_heads else None,
            "positions": positions, "frequencies": frequencies, "amplitude": amplitude}


def _frequencies(case):
    """Radians a position of each pair (float64) and the factor on the turned elements."""
    n, base, s = case["dims"], case["base"], case["factor"]
    if case["method"] == "base":
        base = base * s ** (n / (n - 2))
    f = torch.tensor([base ** (-2.0 * i / n) for i in range(n // 2)], dtype=torch.float64, device=DEVICE)
    if case["method"] == "positions":
        f = f / s
    if case["method"] != "parts":
        return f, 1.0
    # pairs that turn more than 32 times within the original 8192 positions keep their frequency,
    # those that turn less than once have it divided
    kept = ((f * 8192 / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
    return f * kept + f / s * (1.0 - kept), 0.1 * math.log(s) + 1.0


def _prepare_route(case, gen):
    tokens, experts = case["tokens"], case["experts"]
    # some experts are preferred, and the bias works against that
    liked = 0.7 * torch.randn(experts, generator=gen, device=DEVICE)
    logits = (liked + 1.5 * torch.randn((tokens, experts), generator=gen, device=DEVICE)).to(_dtype(case))
    bias = None
    if case["bias"]:
        bias = -0.1 * liked + 0.02 * torch.randn(experts, generator=gen, device=DEVICE)
    return {"case": case, "logits": logits, "bias": bias}


def _prepare_rows(case, gen):
    tokens, experts, k, hidden = (case[n] for n in ("tokens", "experts", "top_k", "hidden"))
    liked = 0.5 * torch.randn(experts, generator=gen, device=DEVICE)
    scores = liked + torch.randn((tokens, experts), generator=gen, device=DEVICE)
    best = scores.topk(k, 1)
    weights = torch.softmax(best.values, 1)
    x = torch.randn((tokens, hidden), generator=gen, device=DEVICE).bfloat16()
    # what the experts gave for each row, in their order
    y = torch.randn((tokens * k, hidden), generator=gen, device=DEVICE).to(_dtype(case))
    add = torch.randn((tokens, hidden), generator=gen, device=DEVICE).bfloat16() if case["add"] else None
    return {"case": case, "x": x, "experts": best.indices.int(), "weights": weights, "y": y, "add": add}


def _lengths(case):
    """Queries and keys of each sequence: spread evenly from short to long, and what is cached before them."""
    b, short, long = case["batch"], case["short"], case["long"]
    q = [long - (long - short) * i // max(1, b - 1) for i in range(b)]
    # neighbours of different lengths
    q = q[::2] + q[1::2][::-1]
    return q, [n + case["cached"] - (case["cached"] // 5) * (i % 3) for i, n in enumerate(q)]


def _starts(lengths):
    starts = [0]
    for n in lengths:
        starts.append(starts[-1] + n)
    return starts


def _prepare_prompt(case, gen):
    heads, kv_heads, d = case["heads"], case["kv_heads"], case["head_dim"]
    q_lens, k_lens = _lengths(case)
    q_starts, k_starts = _starts(q_lens), _starts(k_lens)
    qkv = _projected(gen, q_starts[-1], heads + 2 * kv_heads, d).bfloat16()
    if case["cached"]:
        k, v = (_projected(gen, k_starts[-1], kv_heads, d).bfloat16() for _ in range(2))
    else:
        k, v = qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:]
    offsets = [torch.tensor(s, dtype=torch.int32, device=DEVICE) for s in (q_starts, k_starts)]
    return {"case": case, "q": qkv[:, :heads], "k": k, "v": v, "q_offsets": offsets[0],
            "k_offsets": offsets[1] if case["cached"] else None}


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    make = {"rotary": _prepare_rotary, "route": _prepare_route, "rows": _prepare_rows, "prompt": _prepare_prompt}
    return make[case["op"]](case, gen)


# ---- one pass --------------------------------------------------------------

def _plain_rotary(state):
    case, amplitude = state["case"], state["amplitude"]
    angle = state["positions"].double()[:, None] * state["frequencies"]
    cos, sin = (t.float()[:, None] for t in (torch.cos(angle) * amplitude, torch.sin(angle) * amplitude))
    if case["inverse"]:
        sin = -sin

    def turned(x):
        if x is None:
            return None
        n, y = case["dims"], x.float().clone()
        a, b = (slice(0, n, 2), slice(1, n, 2)) if case["interleaved"] else (slice(0, n // 2), slice(n // 2, n))
        xa, xb = y[..., a].clone(), y[..., b].clone()
        y[..., a] = xa * cos - xb * sin
        y[..., b] = xb * cos + xa * sin
        return y.to(x.dtype)

    return tuple(t for t in (turned(state["q"]), turned(state["k"])) if t is not None)


def _plain_route(state):
    case, x = state["case"], state["logits"].double()
    tokens, experts, k, groups = (case[n] for n in ("tokens", "experts", "top_k", "groups"))
    if case["scoring"] == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    # without a bias the logits are in the scores' order, and exact
    key = x if state["bias"] is None else score + state["bias"].double()
    if groups > 1:
        of_score = score if state["bias"] is None else key
        best = of_score.view(tokens, groups, -1).sort(-1, descending=True).values[..., :2].sum(-1)
        open_ = torch.zeros_like(best, dtype=torch.bool)
        open_.scatter_(1, best.sort(dim=1, descending=True, stable=True).indices[:, :case["top_groups"]], True)
        key = key.masked_fill(~open_.repeat_interleave(experts // groups, 1), float("-inf"))
    chosen = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, chosen)
    if case["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    return (w * case["scale"]).float(), chosen.int()


def _plain_rows(state):
    case, experts = state["case"], state["experts"]
    tokens, k = case["tokens"], case["top_k"]
    flat = experts.reshape(-1).long()
    order = flat.sort(dim=0, stable=True).indices  # row -> token * k + choice
    counts = torch.zeros(case["experts"], dtype=torch.int64, device=flat.device).index_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    place = torch.empty_like(flat)
    place[order] = torch.arange(tokens * k, device=flat.device)
    rows = state["x"][order // k]
    place = place.view(tokens, k)
    total = (state["weights"][..., None] * state["y"][place].float()).sum(1)
    if state["add"] is not None:
        total = total + state["add"].float()
    return rows, offsets, place.int(), total.bfloat16()


def _plain_prompt(state):
    case, q = state["case"], state["q"]
    kv_heads, d = case["kv_heads"], case["head_dim"]
    q_off = state["q_offsets"].long()
    k_off = q_off if state["k_offsets"] is None else state["k_offsets"].long()
    m, n = (torch.diff(t)[:, None] for t in (q_off, k_off))  # lengths
    # the sequences laid out one below the other, padded to the longest
    q_lens, k_lens = _lengths(case)
    at_q, at_k = (torch.arange(max(t), device=q.device) for t in (q_lens, k_lens))
    rows = q.float()[(q_off[:-1, None] + at_q).clamp(max=sum(q_lens) - 1)]
    rows = rows.view(*rows.shape[:2], kv_heads, -1, d).permute(0, 2, 3, 1, 4)  # [batch, kv_heads, heads of each, q, d]
    at = (k_off[:-1, None] + at_k).clamp(max=sum(k_lens) - 1)
    k, v = (state[x].float()[at].transpose(1, 2) for x in ("k", "v"))
    s = torch.matmul(rows.flatten(2, 3) * d ** -0.5, k.transpose(2, 3).contiguous())
    s = s.view(*rows.shape[:-1], -1)
    hidden = at_k > (at_q + n - m)[..., None]  # [batch, q, k]
    s.masked_fill_(hidden[:, None, None], float("-inf"))
    s.sub_(s.amax(-1, keepdim=True)).exp_()
    s.div_(s.sum(-1, keepdim=True))
    o = torch.matmul(s.flatten(2, 3), v.contiguous()).view(rows.shape)
    return o.permute(0, 3, 1, 2, 4).flatten(2, 3)[at_q < m].bfloat16()


def _own(state):
    import fp4_block_quantization_amd as fq
    case = state["case"]
    if case["op"] == "rotary":
        q, k = fq.rotary(state["q"], state["k"], state["positions"], state["frequencies"],
                         amplitude=state["amplitude"], interleaved=case["interleaved"], inverse=case["inverse"])
        return (q,) if k is None else (q, k)
    if case["op"] == "route":
        return fq.moe_route(state["logits"], case["top_k"], bias=state["bias"], scoring=case["scoring"],
                            groups=case["groups"], top_groups=case["top_groups"],
                            renormalize=case["renormalize"], scale=case["scale"])
    if case["op"] == "rows":
        rows, offsets, place = fq.moe_dispatch(state["x"], state["experts"], case["experts"])
        return rows, offsets, place, fq.moe_combine(state["y"], place, state["weights"], add=state["add"])
    return fq.prompt_attention(state["q"], state["k"], state["v"], state["q_offsets"], state["k_offsets"])


def run(state):
    if own:
        return _own(state)
    plain = {"rotary": _plain_rotary, "route": _plain_route, "rows": _plain_rows, "prompt": _plain_prompt}
    return plain[state["case"]["op"]](state)


# ---- what a pass cannot do without -----------------------------------------

def work(case):
    size = 4 if case.get("dtype") == "f32" else 2
    if case["op"] == "rotary":
        heads = case["heads"] + case["kv_heads"]
        return {"bytes": case["tokens"] * (2.0 * heads * case["head_dim"] * size + 8) + 4 * case["dims"],
                "flops": case["tokens"] * (3.0 * heads * case["dims"] + 10.0 * case["dims"])}
    if case["op"] == "route":
        tokens, experts, k = case["tokens"], case["experts"], case["top_k"]
        return {"bytes": tokens * (experts * float(size) + 8 * k) + (4 * experts if case["bias"] else 0),
                "flops": 4.0 * tokens * experts}
    if case["op"] == "rows":
        tokens, k, hidden = case["tokens"], case["top_k"], case["hidden"]
        return {"bytes": tokens * hidden * (2.0 + 2 * k + size * k + 2 + (2 if case["add"] else 0))
                + tokens * k * 12.0 + 8 * case["experts"], "flops": 2.0 * tokens * k * hidden}
    q_lens, k_lens = _lengths(case)
    heads, kv_heads, d = case["heads"], case["kv_heads"], case["head_dim"]
    seen = sum(m * (n - m) + m * (m + 1) // 2 for m, n in zip(q_lens, k_lens))
    return {"bytes": 4.0 * sum(q_lens) * heads * d + 4.0 * sum(k_lens) * kv_heads * d + 8.0 * case["batch"],
            "flops": 4.0 * heads * d * seen + 1.0}


# ---- the definitions in 64 bits --------------------------------------------

def _exact_rotary(state, case):
    n = case["dims"]
    pair = torch.arange(n // 2, dtype=torch.float64, device=DEVICE)
    base = case["base"] * (case["factor"] ** (n / (n - 2.0)) if case["method"] == "base" else 1.0)
    radians = torch.exp(pair * (-2.0 / n * math.log(base)))
    gain = 1.0
    if case["method"] == "positions":
        radians = radians / case["factor"]
    elif case["method"] == "parts":
        turns = radians * (8192 / (2 * math.pi))
        share = torch.where(turns < 1, torch.zeros_like(turns),
                            torch.where(turns > 32, torch.ones_like(turns), (turns - 1) / 31))
        radians = (1 - share) * radians / case["factor"] + share * radians
        gain = 1.0 + math.log(case["factor"]) / 10
    turn = torch.polar(torch.full((), gain, dtype=torch.float64, device=DEVICE),
                       state["positions"].double()[:, None, None] * (-radians if case["inverse"] else radians))
    outs = []
    for x in (state["q"], state["k"]):
        if x is None:
            continue
        x = x.double()
        part = x[..., :n].unflatten(-1, (n // 2, 2) if case["interleaved"] else (2, n // 2))
        pairs = part if case["interleaved"] else part.transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z if case["interleaved"] else z.transpose(-1, -2)
        outs.append(torch.cat([z.flatten(-2), x[..., n:]], -1))
    return tuple(outs)


def _exact_route(state, case):
    x = state["logits"].double()
    score = torch.softmax(x, 1) if case["scoring"] == "softmax" else torch.sigmoid(x)
    bias = None if state["bias"] is None else state["bias"].double()
    key = x.clone() if bias is None else score + bias
    at = torch.arange(case["experts"], device=x.device)
    if case["groups"] > 1:
        # open the groups with the largest sum of their two best, one at a time, the lowest index first
        of = score if bias is None else key
        split = of.reshape(case["tokens"], case["groups"], -1)
        first = split.amax(-1)
        again = split.clone()
        at_first = (split == first[..., None]).to(torch.int8).argmax(-1, keepdim=True)
        again.scatter_(-1, at_first, float("-inf"))
        total = first + again.amax(-1)
        shut = torch.ones_like(total, dtype=torch.bool)
        for _ in range(case["top_groups"]):
            left = total.masked_fill(~shut, float("-inf"))
            pick = (left == left.amax(1, keepdim=True)).to(torch.int8).argmax(1, keepdim=True)
            shut.scatter_(1, pick, False)
        key = torch.where(shut.gather(1, (at // (case["experts"] // case["groups"])).expand_as(key)),
                          torch.full_like(key, float("-inf")), key)
    chosen = []
    for _ in range(case["top_k"]):
        pick = torch.where(key == key.amax(1, keepdim=True), at, case["experts"]).amin(1, keepdim=True)
        chosen.append(pick)
        key = key.scatter(1, pick, float("-inf"))
    chosen = torch.cat(chosen, 1)
    w = score.gather(1, chosen)
    if case["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    return w * case["scale"], chosen.int()


def _exact_rows(state, case):
    tokens, k = case["tokens"], case["top_k"]
    flat = state["experts"].reshape(-1).long()
    # rows by expert, then token: distinct keys
    key = flat * (tokens * k) + torch.arange(tokens * k, device=flat.device)
    order = key.argsort()
    offsets = torch.searchsorted(flat[order], torch.arange(case["experts"] + 1, device=flat.device))
    place = order.argsort().reshape(tokens, k)
    total = (state["y"].double()[place] * state["weights"].double()[..., None]).sum(1)
    if state["add"] is not None:
        total = total + state["add"].double()
    return state["x"].double()[order // k], offsets, place.int(), total


def _exact_prompt(state, case):
    heads, kv_heads, d = case["heads"], case["kv_heads"], case["head_dim"]
    q_lens, k_lens = _lengths(case)
    outs, q0, k0 = [], 0, 0
    for m, n in zip(q_lens, k_lens):
        o = torch.zeros((m, heads, d), dtype=torch.float64, device=DEVICE)
        for h in range(heads):
            k, v = (state[x][k0:k0 + n, h * kv_heads // heads].double() for x in ("k", "v"))
            for a in range(0, m, 2048):
                b = min(a + 2048, m)
                seen = n - m + b  # keys that any of these queries sees
                s = (state["q"][q0 + a:q0 + b, h].double() / math.sqrt(d)) @ k[:seen].t()
                late = torch.ones_like(s, dtype=torch.bool).triu(n - m + a + 1)
                o[a:b, h] = torch.softmax(s.masked_fill(late, float("-inf")), 1) @ v[:seen]
        outs.append(o)
        q0, k0 = q0 + m, k0 + n
    return torch.cat(outs)


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(state, case)
    if case["op"] == "route":
        return _exact_route(state, case)
    return _exact_rows(state, case) if case["op"] == "rows" else _exact_prompt(state, case)
