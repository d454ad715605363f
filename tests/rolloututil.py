"""References for the rollout operators' tests: 4-bit tensors decoded to
float64 by table, products and attention in float64 on the CPU, and the
error bounds of the kernels' arithmetic."""
import math

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
SIGNED = np.concatenate([GRID, -GRID])


def e4m3(b):
    b = np.asarray(b, np.int64)
    ex, frac = (b >> 3) & 15, b & 7
    v = np.where(ex > 0, (8 + frac) * 2.0 ** (ex - 10), frac * 2.0 ** -9)
    v = np.where((b & 0x7F) == 0x7F, np.nan, v)
    return np.where(b & 0x80, -v, v)


def unpack(codes):
    n = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    return SIGNED[n]


def nv_values(codes, scales, s):
    """float64 [..., d] of codes u8 [..., d/2], E4M3 bytes [..., d/16], s [...]."""
    return unpack(codes) * np.repeat(e4m3(scales), 16, -1) * np.asarray(s, np.float64)[..., None]


def mx_values(codes, scales):
    return unpack(codes) * np.repeat(2.0 ** (np.asarray(scales, np.float64) - 127), 32, -1)


def bf16_values(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def linear_bound(x, w, out_bf16):
    """Elementwise bound on |y - x.w^T|: k additions in FP32, each off by at
    most 2^-23 of the running sum of magnitudes (truncation allowed for), the
    block and row scale products, activations below 2^-39 of their row's
    largest taken as zero, and one rounding to BF16."""
    k = x.shape[1]
    mag = np.abs(x) @ np.abs(w).T
    b = (k + 8) * 2.0 ** -23 * mag
    b += 2.0 ** -39 * np.abs(x).max(1, initial=0)[:, None] * np.abs(w).sum(1)[None, :]
    y = x @ w.T
    return y, b + (2.0 ** -8 * np.abs(y) if out_bf16 else 0) + 1e-37


def attention(q, k, v, scale):
    """(o, lse, bound, lse bound) for q [h, d], k and v [t, h, d] already per query head,
    in float64.  bound: FP32 scores (d additions, each 2^-23 of the sum of
    magnitudes, and as much again for the softmax's own FP32 steps), an FP16
    rounding of each probability (2^-11), probabilities below 2^-38 of the
    largest value scale lost, and the output's rounding to BF16."""
    h, d = q.shape
    t = k.shape[0]
    if t == 0:
        return np.zeros((h, d)), np.full(h, -math.inf), np.zeros((h, d)), np.zeros(h)
    s = np.einsum("hd,thd->ht", q, k) * scale
    mag = np.einsum("hd,thd->ht", np.abs(q), np.abs(k)) * abs(scale)
    top = s.max(1, keepdims=True)
    p = np.exp(s - top)
    l = p.sum(1, keepdims=True)
    p = p / l
    o = np.einsum("ht,thd->hd", p, v)
    delta = (d + 32) * 2.0 ** -23 * (mag.max(1) + 1.0)
    spread = np.einsum("ht,thd->hd", p, np.abs(v))
    b = spread * (2.0 ** -10 + 4 * delta + (t + 8) * 2.0 ** -23)[:, None]
    b += t * 2.0 ** -38 * np.abs(v).max() + 2.0 ** -8 * np.abs(o) + 1e-37
    return o, (top + np.log(l))[:, 0], b, 2 * delta + (t + 8) * 2.0 ** -23 + 2.0 ** -20


def check(got, want, bound, label):
    got = np.asarray(got, np.float64)
    assert np.isfinite(got).all(), "%s: not finite" % label
    over = np.abs(got - want) - bound
    if over.size and over.max() > 0:
        i = np.unravel_index(np.argmax(over), over.shape)
        raise AssertionError("%s: at %s got %r want %r, bound %.3g (%d of %d outside)" % (
            label, i, got[i], want[i], bound[i], int((over > 0).sum()), over.size))
