"""References for the tests of the operators in include/fp4q/layer.h, in
float64 on the CPU, and the error bounds of the kernels' arithmetic.  A
rounding is off by half a step: 2^-24 of an FP32 value, 2^-8 of a BF16 one."""
import math

import numpy as np

BF16, FP32 = 2.0 ** -8, 2.0 ** -24


def f64(t):
    return t.detach().double().cpu().numpy()


def rotary(x, positions, frequencies, amplitude, interleaved, inverse, bf16):
    """x float64 [tokens, heads, d] turned, and a bound on the kernel's error.
    Sine and cosine are within 2^-23, their product with the amplitude, the two
    products and their sum round (FP32), then the result; the angle itself, in
    FP64, is known to 2^-52 of its size on both sides."""
    n = 2 * len(frequencies)
    angle = positions.astype(np.float64)[:, None, None] * frequencies
    c, s = np.cos(angle) * amplitude, np.sin(angle) * amplitude * (-1 if inverse else 1)
    a, b = (slice(0, n, 2), slice(1, n, 2)) if interleaved else (slice(0, n // 2), slice(n // 2, n))
    y, bound = x.copy(), np.zeros_like(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    mag = (np.abs(x[..., a]) + np.abs(x[..., b])) * abs(amplitude)
    off = mag * (2.0 ** -23 + 4 * FP32 + np.abs(angle) * 2.0 ** -51)
    bound[..., a] = off + (BF16 * (np.abs(y[..., a]) + off) if bf16 else 0)
    bound[..., b] = off + (BF16 * (np.abs(y[..., b]) + off) if bf16 else 0)
    return y, bound + 1e-44  # (FP32's smallest step)


def prompt(q, k, v, scale):
    """Causal attention of one sequence, q [m, h, d], k and v [n, h, d] already per query
    head, queries the last of the keys: (o, lse, bound, lse bound).  Scores: d
    additions in FP32, each off by at most 2^-23 of the sum of magnitudes (truncation
    allowed for), and as much for the exponent's own steps; a BF16 rounding of every
    probability; the sums; the result's rounding to BF16."""
    m, h, d = q.shape
    n = k.shape[0]
    o, bound = np.zeros((m, h, d)), np.zeros((m, h, d))
    lse, lse_bound = np.full((m, h), -math.inf), np.zeros((m, h))
    if n == 0:
        return o, lse, bound, lse_bound
    hidden = np.arange(n)[None, :] > (n - m + np.arange(m))[:, None]
    for i in range(h):
        s = (q[:, i] @ k[:, i].T) * scale
        mag = (np.abs(q[:, i]) @ np.abs(k[:, i]).T) * abs(scale)
        s[hidden], mag[hidden] = -math.inf, 0.0
        top = s.max(1, keepdims=True)
        some = np.isfinite(top[:, 0])
        p = np.exp(s - np.where(np.isfinite(top), top, 0.0))
        l = p.sum(1, keepdims=True)
        p = p / np.where(l > 0, l, 1.0)
        o[:, i] = p @ v[:, i]
        delta = (d + 32) * 2.0 ** -23 * (mag.max(1) + 1.0)
        spread = p @ np.abs(v[:, i])
        b = spread * (BF16 + 4 * delta + (n + 8) * 2.0 ** -23)[:, None]
        bound[:, i] = b + BF16 * (np.abs(o[:, i]) + b) + 1e-37
        lse[some, i] = (top[:, 0] + np.log(np.where(l > 0, l, 1.0))[:, 0])[some]
        lse_bound[:, i] = 2 * delta + (n + 8) * 2.0 ** -23 + np.abs(np.where(some, lse[:, i], 0)) * 2.0 ** -22
    return o, lse, bound, lse_bound


def route(logits, top_k, bias, scoring, groups, top_groups, renormalize, scale):
    """(weights, experts) of float64 logits [tokens, experts], token by token."""
    tokens, experts = logits.shape
    weights, chosen = np.zeros((tokens, top_k)), np.zeros((tokens, top_k), np.int64)
    for t in range(tokens):
        x = logits[t]
        if scoring == "sigmoid":
            with np.errstate(over="ignore"):
                score = 1.0 / (1.0 + np.exp(-x))
        elif x.max() == -math.inf:
            score = np.zeros(experts)
        else:
            score = np.exp(x - x.max())
            score = score / score.sum()
        key = (x if bias is None else score + bias).copy()
        if groups > 1:
            marks = score if bias is None else key
            per = experts // groups
            mark = [sum(sorted(marks[g * per:(g + 1) * per])[-2:]) for g in range(groups)]
            best = sorted(range(groups), key=lambda g: (-mark[g], g))[:top_groups]
            allowed = [e for e in range(experts) if e // per in best]
        else:
            allowed = range(experts)
        order = sorted(allowed, key=lambda e: (-key[e], e))[:top_k]
        w = score[order]
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else np.zeros(top_k)
        weights[t], chosen[t] = w * scale, order
    return weights, chosen


def dispatch(experts, num_experts):
    """offsets and place of [tokens, top_k] experts: by expert, then token, then choice."""
    flat = experts.reshape(-1)
    ok = (flat >= 0) & (flat < num_experts)
    counts = np.bincount(flat[ok], minlength=num_experts)
    order = np.argsort(np.where(ok, flat, num_experts), kind="stable")[:ok.sum()]
    place = np.full(flat.shape, -1)
    place[order] = np.arange(len(order))
    return np.concatenate([[0], counts.cumsum()]), place.reshape(experts.shape)


def check(got, want, bound, label):
    got = np.asarray(got, np.float64)
    assert got.shape == want.shape, label
    assert np.isfinite(got).all(), "%s: not finite" % label
    over = np.abs(got - want) - bound
    if over.size and over.max() > 0:
        i = np.unravel_index(np.argmax(over), over.shape)
        raise AssertionError("%s: at %s got %r want %r, bound %.3g (%d of %d outside)" % (
            label, i, got[i], want[i], np.broadcast_to(bound, over.shape)[i], int((over > 0).sum()),
            over.size))
