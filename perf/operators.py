"""The rollout-serving operators, measured: their cases, their plain forms in
elementary torch operations (FP32, rounded once at the end) and the calls a
user makes of them.

Three operators of a 4-bit rollout engine:
  linear     y = x . DQ(W)^T for weights held in NVFP4 (16-element E4M3 block
             scales and an FP32 scale per output row) or MXFP4 (32-element
             E8M0 scales), for one matrix or for experts with routed rows
  cache      keys and values quantized to NVFP4 as they are written to a
             paged cache, and read back as BF16
  attention  softmax attention over that cache, for one or a few new tokens
             per sequence, optionally over a prefix that a group of sequences
             shares in front of each one's own tokens

Cache layout (one row = the head_dim elements of one token and head):
  k_codes u8 [pages, kv_heads, page, d/2]   v_codes u8 [pages, kv_heads, page, d/2]
  k_scales u8 [pages, kv_heads, page, d/16] v_scales u8 [pages, kv_heads, d/16, page]
  k_token_scales, v_token_scales f32 [pages, kv_heads, page]
"""
import functools
import math
import operator

import torch

own = False

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DEVICE = "cuda"


# ---- cases -----------------------------------------------------------------

def _linear(name, fmt, rows, n, k, experts=0, out="bf16"):
    return {"name": name, "op": "linear", "format": fmt, "rows": rows, "n": n, "k": k,
            "experts": experts, "out": out}


def _cache(name, batch, cached, new, kv_heads, head_dim, page, whole, four_over_six=True):
    return {"name": name, "op": "cache", "batch": batch, "cached": cached, "new": new,
            "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "whole": whole,
            "four_over_six": four_over_six}


def _attention(name, batch, tokens, heads, kv_heads, head_dim, page, short, long, groups=0,
               prefix=0):
    return {"name": name, "op": "attention", "batch": batch, "tokens": tokens, "heads": heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "short": short,
            "long": long, "groups": groups, "prefix": prefix}


def listed():
    return [
        # one token through one expert's projection: the latency of a single matrix-vector product
        _linear("linear_1x2048x7168", "nv", 1, 2048, 7168),
        # a decode batch of 48 rollouts through one projection back to the hidden size
        _linear("linear_48x7168x2048", "nv", 48, 7168, 2048, out="f32"),
        # 32 tokens routed to 8 of 32 experts each: every expert's weights are read for a few rows
        _linear("linear_experts_256", "nv", 256, 2048, 7168, experts=32),
        # MXFP4 weights, with an odd row count, output width and depth
        _linear("linear_mx_5x1999x1376", "mx", 5, 1999, 1376),
        # a decode step's cache write: one new token for each of 64 sequences
        _cache("cache_decode_64", 64, 1000, 1, 8, 128, 16, False),
        # chunked prefill: a chunk is written behind a cached context, which is read back whole
        _cache("cache_chunk_4x2048", 4, 6001, 2048, 8, 128, 64, True),
        # a few sequences with odd lengths, heads of 80 and scales without Four-Over-Six
        _cache("cache_odd_7x33", 7, 211, 33, 3, 80, 48, True, four_over_six=False),
        # one sequence's decode step at a modest context: latency
        _attention("attention_1x777", 1, 1, 32, 8, 128, 16, 777, 777),
        # a full decode batch with long contexts of mixed length: the largest
        _attention("attention_64x8192", 64, 1, 64, 8, 128, 64, 2048, 8192),
        # three drafted tokens verified at once, ragged lengths from nothing up, small heads
        _attention("attention_13x3x1500", 13, 3, 12, 3, 64, 16, 0, 1500),
        # rollouts of four prompts, sixteen samples each: the prompt is read once for its samples
        _attention("attention_prefix_4x16", 64, 1, 32, 8, 128, 64, 64, 1024, groups=4, prefix=8192),
        # uneven groups with odd prompt lengths and wide heads
        _attention("attention_prefix_3_odd", 11, 2, 10, 2, 256, 32, 1, 333, groups=3, prefix=1777),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear", "cache", "attention", "attention", "prefix"))
    if op == "linear":
        fmt = rng.choice(("nv", "mx"))
        experts = rng.choice((0, 0, rng.randint(2, 32)))
        k = 32 * _log(rng, 2, 224) if fmt == "mx" else 16 * _log(rng, 4, 448)
        return {**_linear("", fmt, _log(rng, 1, 256 if experts else 64), _log(rng, 16, 2048 if experts else 8192), k,
                          experts, rng.choice(("bf16", "f32")))}
    if op == "cache":
        batch = _log(rng, 1, 64)
        return _cache("", batch, _log(rng, 1, max(2, 24000 // batch)), _log(rng, 1, max(2, 8192 // batch)),
                      rng.randint(1, 8), 16 * rng.randint(4, 16), rng.choice((16, 32, 48, 64, 128)),
                      rng.random() < 0.5, rng.random() < 0.7)
    kv_heads = rng.randint(1, 8)
    heads = kv_heads * rng.choice((1, 2, 4, 5, 8))
    batch = _log(rng, 1, 64)
    long = _log(rng, 16, 8192)
    page, head_dim, tokens = rng.choice((16, 32, 64, 128)), rng.choice((64, 128, 128, 192, 256)), rng.choice((1, 1, 1, 2, 4))
    if op == "attention":
        return _attention("", batch, tokens, heads, kv_heads, head_dim if batch * long < 262144 else 128, page,
                          rng.randint(0, long), long)
    return _attention("", batch, tokens, heads, kv_heads, min(head_dim, 128), page, rng.randint(0, min(long, 1024)),
                      min(long, 1024), rng.randint(1, max(1, batch // 3)), _log(rng, 64, 8192))


# ---- quantization in elementary operations (inputs, and the cache's plain form) ----------------

def _signed_grid(device):
    g = torch.tensor(GRID, dtype=torch.float32, device=device)
    return torch.cat([g, -g])


def _nearest(v):
    """E2M1 code of v >= 0, ties to the even code, saturating."""
    return ((v > 0.25).to(torch.uint8) + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5)
            + (v >= 3.5) + (v > 5.0))


def _candidate(blocks, amax, s, k):
    """Scales (E4M3 values), codes and values of blocks [..., n, 16] whose maximum maps to k."""
    step = k * s
    # divisors are tensors throughout: torch multiplies by the rounded reciprocal of a plain number
    e = torch.where(step > 0, amax / step, torch.zeros_like(amax)).clamp(max=448.0)
    e = e.to(torch.float8_e4m3fn).float()
    d = e * s
    r = torch.where(d > 0, torch.ones_like(d) / d, torch.zeros_like(d))[..., None]
    code = _nearest(blocks.abs() * r)
    c = (_signed_grid(blocks.device)[code.long()] * e[..., None]) * s[..., None]
    return e, code, torch.where(blocks < 0, -c, c)


def _error(x, c):
    """Squared error of each block, summed in element order (the choice between candidates is on it)."""
    d = x - c
    return functools.reduce(operator.add, (d * d).unbind(-1))


def _nv_rows(x, four_over_six):
    """NVFP4 of FP32 rows [..., d]: nibbles u8 [..., d], E4M3 values [..., d/16], row scales [...]."""
    blocks = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    amax = blocks.abs().amax(-1)
    top = amax.amax(-1, keepdim=True)
    s = top / torch.full_like(top, 1536.0 if four_over_six else 2688.0)
    e, code, c = _candidate(blocks, amax, s, 6.0)
    if four_over_six:
        e4, code4, c4 = _candidate(blocks, amax, s, 4.0)
        four = _error(blocks, c4) < _error(blocks, c)
        e, code = torch.where(four, e4, e), torch.where(four[..., None], code4, code)
    nibble = code | (torch.signbit(blocks).to(torch.uint8) << 3)
    return nibble.reshape(x.shape), e, s[..., 0]


def _pack(nibbles):
    return nibbles[..., 0::2] | (nibbles[..., 1::2] << 4)


def _unpack(codes):
    """Signed E2M1 values (FP32) of packed codes, low nibble first."""
    n = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    return _signed_grid(codes.device)[n.long()]


def _e4m3(scales):
    return scales.view(torch.float8_e4m3fn).float()


def _nv_values(codes, e, s):
    """FP32 values of packed codes [..., d/2], E4M3 values [..., d/16] and row scales [...]."""
    g = _unpack(codes)
    g = g.reshape(*g.shape[:-1], e.shape[-1], 16) * e[..., None]
    return (g * s[..., None, None]).flatten(-2)


# ---- inputs ----------------------------------------------------------------

def _weights(gen, case):
    """Codes and scales of experts x n x k weights, quantized matrix by matrix."""
    experts, n, k = max(1, case["experts"]), case["n"], case["k"]
    parts = []
    for _ in range(experts):
        w = 0.02 * torch.randn((n, k), generator=gen, device=DEVICE)
        if case["format"] == "nv":
            nib, e, s = _nv_rows(w.bfloat16().float(), True)
            parts.append((_pack(nib), e.to(torch.float8_e4m3fn).view(torch.uint8), s))
        else:
            b = w.bfloat16().float().reshape(n, k // 32, 32)
            top = b.abs().amax(-1).clamp(min=2.0 ** -120)
            ex = torch.floor(torch.log2(top)) - 2
            code = _nearest(b.abs() * torch.exp2(-ex)[..., None])
            nib = code | (torch.signbit(b).to(torch.uint8) << 3)
            parts.append((_pack(nib.reshape(n, k)), (ex + 127).to(torch.uint8)))
    stacked = [torch.stack(t) for t in zip(*parts)]
    return stacked if case["experts"] else [t[0] for t in stacked]


def _prepare_linear(case, gen):
    rows, k, experts = case["rows"], case["k"], case["experts"]
    # activations with per-token gains and a few outlier channels
    x = torch.randn((rows, k), generator=gen, device=DEVICE)
    x = x * torch.exp(0.5 * torch.randn((rows, 1), generator=gen, device=DEVICE))
    x[:, torch.randperm(k, generator=gen, device=DEVICE)[:max(1, k // 200)]] *= 30.0
    state = {"case": case, "x": x.bfloat16(), "w": _weights(gen, case), "offsets": None}
    if experts:
        to = torch.randint(0, experts, (rows,), generator=gen, device=DEVICE)
        counts = torch.zeros(experts, dtype=torch.int64, device=DEVICE).index_add_(0, to, torch.ones_like(to))
        state["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return state


def _keys(gen, *shape):
    """Keys or values as a projection leaves them: per-token gains and a few strong channels."""
    x = torch.randn(shape, generator=gen, device=DEVICE)
    x *= torch.exp(0.4 * torch.randn((*shape[:-1], 1), generator=gen, device=DEVICE))
    x[..., torch.randperm(shape[-1], generator=gen, device=DEVICE)[:max(1, shape[-1] // 32)]] *= 4.0
    return x.bfloat16()


def _filled(gen, pages, case):
    """A paged cache full of quantized rows, made a slice of pages at a time."""
    h, p, d = case["kv_heads"], case["page"], case["head_dim"]
    step, parts = max(1, (1 << 25) // (h * p * d)), []
    for a in range(0, pages, step):
        n = min(step, pages - a)
        part = []
        for value in (False, True):
            nib, e, s = _nv_rows(_keys(gen, n, h, p, d).float(), case.get("four_over_six", True))
            e = e.to(torch.float8_e4m3fn).view(torch.uint8)
            part += [_pack(nib), e.transpose(2, 3).contiguous() if value else e, s]
        parts.append(part)
    return [torch.cat(t) for t in zip(*parts)]


def _table(gen, rows, per_row, pages):
    """[rows, per_row] page ids, a shuffled part of the cache."""
    return torch.randperm(pages, generator=gen, device=DEVICE)[:rows * per_row].reshape(rows, per_row)


def _slots(table, page, start, count):
    """Slots (page * page_size + place) of tokens start..start+count of each row's sequence."""
    at = torch.arange(start, start + count, device=DEVICE)
    return (table[:, at // page] * page + at % page).reshape(-1)


def _prepare_cache(case, gen):
    batch, cached, new, page = case["batch"], case["cached"], case["new"], case["page"]
    per = -(-(cached + new) // page)
    pages = batch * per + 3
    table = _table(gen, batch, per, pages)
    return {"case": case, "cache": _filled(gen, pages, case),
            "k": _keys(gen, batch * new, case["kv_heads"], case["head_dim"]),
            "v": _keys(gen, batch * new, case["kv_heads"], case["head_dim"]),
            "slots": _slots(table, page, cached, new),
            "back": _slots(table, page, 0, cached + new) if case["whole"] else _slots(table, page, cached, new)}


def _lengths(case):
    """Own tokens of each sequence: spread evenly from short to long."""
    b = case["batch"]
    return [case["long"] - (case["long"] - case["short"]) * i // max(1, b - 1) for i in range(b)]


def _prefixes(case):
    """Prefix tokens of each group: the longest, then each a seventh shorter, over again."""
    return [case["prefix"] - (case["prefix"] // 7) * (i % 3) for i in range(case["groups"])]


def _members(case):
    """Sequences of each group: even shares, the first ones one larger."""
    g, b = case["groups"], case["batch"]
    return [b // g + (i < b % g) for i in range(g)]


def _prepare_attention(case, gen):
    batch, page, groups = case["batch"], case["page"], case["groups"]
    per, per_prefix = max(1, -(-case["long"] // page)), -(-case["prefix"] // page)
    pages = batch * per + groups * per_prefix + 3
    lens = torch.tensor(_lengths(case), device=DEVICE)
    ids = _table(gen, 1, batch * per + groups * per_prefix, pages)[0].int()
    state = {"case": case, "cache": _filled(gen, pages, case),
             "q": (2.0 * torch.randn((batch, case["tokens"], case["heads"], case["head_dim"]), generator=gen,
                                     device=DEVICE)).bfloat16(),
             "table": ids[:batch * per].reshape(batch, per).contiguous(),
             "lens": lens[torch.randperm(batch, generator=gen, device=DEVICE)].int(), "prefix": None}
    if groups:
        members = torch.tensor([0] + _members(case), device=DEVICE).cumsum(0).int()
        state["prefix"] = (ids[batch * per:].reshape(groups, per_prefix).contiguous(),
                           torch.tensor(_prefixes(case), device=DEVICE).int(), members)
    return state


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    make = {"linear": _prepare_linear, "cache": _prepare_cache, "attention": _prepare_attention}
    return make[case["op"]](case, gen)


# ---- one pass --------------------------------------------------------------

def _plain_linear(state):
    case, w = state["case"], state["w"]
    x = state["x"].float()
    if case["format"] == "nv":
        dq = _nv_values(w[0], _e4m3(w[1]), w[2])
    else:
        g = _unpack(w[0])
        dq = (g.reshape(*w[1].shape, 32) * torch.exp2(w[1].float() - 127.0)[..., None]).reshape(g.shape)
    if case["experts"]:
        # every row against its own expert's matrix: the rows laid out expert by expert, padded
        off = state["offsets"]
        at = torch.arange(case["rows"], device=x.device)
        expert = torch.searchsorted(off[1:].contiguous(), at, right=True)
        place = at - off[expert]
        padded = x.new_zeros((case["experts"], case["rows"], case["k"]))
        padded[expert, place] = x
        y = torch.matmul(padded, dq.transpose(1, 2))[expert, place]
    else:
        y = x @ dq.t()
    return y if case["out"] == "f32" else y.bfloat16()


def _plain_cache(state):
    case = state["case"]
    page, outs = case["page"], []
    for i, rows in ((0, state["k"]), (3, state["v"])):
        codes, scales, ts = state["cache"][i:i + 3]
        nib, e, s = _nv_rows(rows.float(), case["four_over_six"])
        e = e.to(torch.float8_e4m3fn).view(torch.uint8)
        pg, at = state["slots"] // page, state["slots"] % page
        codes[pg, :, at] = _pack(nib)
        ts[pg, :, at] = s
        if i:
            scales[pg, :, :, at] = e
        else:
            scales[pg, :, at] = e
        pg, at = state["back"] // page, state["back"] % page
        e = scales[pg, :, :, at] if i else scales[pg, :, at]
        outs.append(_nv_values(codes[pg, :, at], _e4m3(e), ts[pg, :, at]).bfloat16())
    return tuple(outs)


def _gathered(cache, table, page, which):
    """FP32 keys (which 0) or values (which 3) of the tables' pages: [rows, heads, tokens, d]."""
    codes, scales, ts = (t[table.long()] for t in cache[which:which + 3])
    e = _e4m3(scales.transpose(-1, -2).contiguous() if which else scales)
    x = _nv_values(codes, e, ts)
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attention(state):
    case = state["case"]
    b, t, h, hk, d = (case[n] for n in ("batch", "tokens", "heads", "kv_heads", "head_dim"))
    q = state["q"].float().reshape(b, t, hk, h // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)
    k, v = (_gathered(state["cache"], state["table"], case["page"], w) for w in (0, 3))
    own_tokens = k.shape[2]
    # token i of t sees its sequence's first length - t + 1 + i tokens
    seen = state["lens"][:, None] - t + 1 + torch.arange(t, device=q.device)
    mask = torch.arange(own_tokens, device=q.device) < seen[..., None]
    if case["groups"]:
        table, lens, members = state["prefix"]
        group = torch.searchsorted(members[1:].contiguous(), torch.arange(b, device=q.device), right=True)
        pk, pv = (_gathered(state["cache"], table, case["page"], w)[group] for w in (0, 3))
        k, v = torch.cat([pk, k], 2), torch.cat([pv, v], 2)
        before = torch.arange(pk.shape[2], device=q.device) < lens[group][:, None]
        mask = torch.cat([before[:, None].expand(b, t, -1), mask], 2)
    scores = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(d)
    scores = scores.reshape(b, hk, h // hk, t, -1).masked_fill(~mask[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    o = torch.matmul(p.reshape(b, hk, -1, p.shape[-1]), v).reshape(b, hk, h // hk, t, d)
    return o.permute(0, 3, 1, 2, 4).reshape(b, t, h, d).bfloat16()


def _own(state):
    import fp4_block_quantization_amd as fq
    case = state["case"]
    if case["op"] == "linear":
        dtype = torch.float32 if case["out"] == "f32" else torch.bfloat16
        call = fq.nvfp4_linear if case["format"] == "nv" else fq.mxfp4_linear
        return call(state["x"], *state["w"], offsets=state["offsets"], out_dtype=dtype)
    if case["op"] == "cache":
        fq.nvfp4_kv_append(state["cache"], state["k"], state["v"], state["slots"],
                           four_over_six=case["four_over_six"])
        return fq.nvfp4_kv_read(state["cache"], state["back"])
    return fq.nvfp4_kv_attention(state["q"], state["cache"], state["table"], state["lens"],
                                 prefix=state["prefix"])


def run(state):
    if own:
        return _own(state)
    plain = {"linear": _plain_linear, "cache": _plain_cache, "attention": _plain_attention}
    return plain[state["case"]["op"]](state)


# ---- what a pass cannot do without -----------------------------------------

def work(case):
    if case["op"] == "linear":
        m, n, k, e = case["rows"], case["n"], case["k"], case["experts"]
        used = e * (1.0 - (1.0 - 1.0 / e) ** m) if e else 1.0  # experts that any row is routed to
        weight = n * (k / 2 + (k / 16 + 4 if case["format"] == "nv" else k / 32))
        return {"bytes": used * weight + 2 * m * k + m * n * (4 if case["out"] == "f32" else 2),
                "flops": 2.0 * m * n * k}
    d, row = case["head_dim"], case["head_dim"] / 2 + case["head_dim"] / 16 + 4
    if case["op"] == "cache":
        new = 2 * case["batch"] * case["new"] * case["kv_heads"]
        back = 2 * case["batch"] * (case["new"] + (case["cached"] if case["whole"] else 0)) * case["kv_heads"]
        return {"bytes": new * (2 * d + row) + back * (row + 2 * d), "flops": 20.0 * new * d + 3.0 * back * d}
    own_tokens, t = sum(_lengths(case)), case["tokens"]
    shared = sum(_prefixes(case))
    seen = own_tokens + sum(p * m for p, m in zip(_prefixes(case), _members(case) if case["groups"] else []))
    return {"bytes": 2.0 * (own_tokens + shared) * case["kv_heads"] * row + 4.0 * case["batch"] * t * case["heads"] * d,
            "flops": 4.0 * t * case["heads"] * seen * d + 1.0}


# ---- the definitions in 64 bits --------------------------------------------

def _exact_decode(codes, e, s=None):
    """Float64 values of packed codes, by table of the 256 bytes; e and s float64 scales."""
    grid = [*GRID, *(-g for g in GRID)]
    pairs = torch.tensor([[grid[b & 15], grid[b >> 4]] for b in range(256)], dtype=torch.float64, device=codes.device)
    x = pairs[codes.int()].flatten(-2)
    x = x * e.repeat_interleave(x.shape[-1] // e.shape[-1], -1)
    return x if s is None else x * s.double()[..., None]


def _exact_e4m3(scales):
    b = scales.int()
    frac, ex = (b & 7).double(), (b >> 3) & 15
    return torch.where(ex > 0, (8 + frac) * torch.exp2(ex.double() - 10), frac * 2.0 ** -9)


def _exact_linear(state):
    case, w = state["case"], state["w"]
    off = state["offsets"].tolist() if case["experts"] else [0, case["rows"]]
    y = torch.zeros((case["rows"], case["n"]), dtype=torch.float64, device=DEVICE)
    for i, (a, b) in enumerate(zip(off, off[1:])):
        part = [t[i] for t in w] if case["experts"] else w
        if case["format"] == "nv":
            m = _exact_decode(part[0], _exact_e4m3(part[1]), part[2])
        else:
            m = _exact_decode(part[0], torch.exp2(part[1].double() - 127))
        y[a:b] = state["x"][a:b].double() @ m.t()
    return y


def _exact_rows(x, four_over_six):
    """Float64 NVFP4 values of rows: scales and codes found by search over the formats' grids."""
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    # row and block scales are what the format stores (FP32 and E4M3): round them there
    blocks = x.double().unflatten(-1, (-1, 16))
    top = blocks.abs().amax(-1)
    s = (top.amax(-1) / (1536 if four_over_six else 2688)).float().double()[..., None]
    every = torch.arange(127, device=x.device)
    scales = _exact_e4m3(every)
    best, best_err = None, None
    for k in ((6, 4) if four_over_six else (6,)):
        t = torch.where(s > 0, top / (k * s), torch.zeros_like(top))
        hi = torch.searchsorted(scales, t.contiguous()).clamp(1, 126)
        lo = hi - 1
        up, down = scales[hi] - t, t - scales[lo]
        e = scales[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)]
        d = (e * s)[..., None]
        v = torch.where(d > 0, blocks.abs() / d, torch.zeros_like(blocks)).clamp(max=6.0)
        hi = torch.searchsorted(grid, v.contiguous()).clamp(1, 7)
        lo = hi - 1
        up, down = grid[hi] - v, v - grid[lo]
        g = grid[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)]
        c = torch.sign(blocks) * g * d
        err = ((blocks - c) ** 2).sum(-1, keepdim=True)
        best, best_err = (c, err) if best is None else (torch.where(err < best_err, c, best), best_err)
    return best.flatten(-2)


def _exact_cache(state):
    case = state["case"]
    page, back, outs = case["page"], state["back"], []
    for i, rows in ((0, state["k"]), (3, state["v"])):
        codes, scales, ts = state["cache"][i:i + 3]
        e = scales.transpose(2, 3) if i else scales
        pg, at = back // page, back % page
        x = _exact_decode(codes[pg, :, at], _exact_e4m3(e[pg, :, at]), ts[pg, :, at])
        # the places that the new tokens take
        order = torch.full((codes.shape[0] * page,), -1, dtype=torch.int64, device=back.device)
        order[state["slots"]] = torch.arange(rows.shape[0], device=back.device)
        new = order[back]
        x[new >= 0] = _exact_rows(rows, case["four_over_six"])[new[new >= 0]]
        outs.append(x)
    return tuple(outs)


def _exact_attention(state):
    case = state["case"]
    t, h, hk, d, page = (case[n] for n in ("tokens", "heads", "kv_heads", "head_dim", "page"))
    out = torch.zeros((case["batch"], t, h, d), dtype=torch.float64, device=DEVICE)
    lens = state["lens"].tolist()
    starts = state["prefix"][2].tolist() if case["groups"] else None

    def tokens(ids, n):
        got = []
        for i in (0, 3):
            codes, scales, ts = (x[ids.long()] for x in state["cache"][i:i + 3])
            e = scales.transpose(2, 3) if i else scales
            x = _exact_decode(codes, _exact_e4m3(e), ts)
            got.append(x.transpose(1, 2).flatten(0, 1)[:n])
        return got

    for b in range(case["batch"]):
        k, v = tokens(state["table"][b], lens[b])
        before = 0
        if starts:
            g = max(i for i in range(case["groups"]) if starts[i] <= b)
            before = int(state["prefix"][1][g])
            pk, pv = tokens(state["prefix"][0][g], before)
            k, v = torch.cat([pk, k]), torch.cat([pv, v])
        for i in range(t):
            n = before + max(0, lens[b] - t + 1 + i)
            if n:
                q = state["q"][b, i].double().reshape(hk, h // hk, d)
                p = torch.softmax(torch.matmul(q, k[:n].permute(1, 2, 0)) / math.sqrt(d), -1)
                out[b, i] = torch.matmul(p, v[:n].transpose(0, 1)).reshape(h, d)
    return out


def exact(case, seed):
    state = prepare(case, seed)
    return {"linear": _exact_linear, "cache": _exact_cache, "attention": _exact_attention}[case["op"]](state)
