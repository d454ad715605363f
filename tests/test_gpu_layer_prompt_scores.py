"""prompt_attention with scores far from zero, of which FP32 holds every one
exactly, against float64 with bounds that a wrong result does not meet; and
sequences beside offsets that are out of range."""
import math

import numpy as np
import pytest
import torch

import fp4_block_quantization_amd as fq
import layerutil as lu

pytestmark = pytest.mark.gpu

DIMS = [64, 128, 192, 256]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.rollout_lib()


def rand(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(shape, generator=g, device="cuda")


def offsets(*lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")


def exact(q, k, v, got, lse, first=0):
    """Every row of one sequence, queries from `first` on.  Scores (scale 1) are whole numbers below
    2^24: exact.  An exponent is a difference of scores times log2 e, whose constant and product
    round (2^-23 of it), and of which no more than 160 counts; the exponential is off by 2 units; a
    probability rounds to BF16; the sums have up to n additions; the result rounds to BF16.  The
    running maximum's moves multiply by further exponentials (8 units for all of them: they are few)."""
    m, n, d = len(q), len(k), q.shape[2]
    rep = q.shape[1] // k.shape[1]
    assert m >= 1 and n >= m
    for h in range(q.shape[1]):
        s = lu.f64(q[:, h]) @ lu.f64(k[:, h // rep]).T
        assert (np.abs(s) < 2 ** 24).all() and (s == np.rint(s)).all()
        s[np.arange(n)[None, :] > (n - m + np.arange(m))[:, None]] = -math.inf
        top = s.max(1, keepdims=True)
        p = np.exp(s - top)
        l = p.sum(1, keepdims=True)
        vv = lu.f64(v[:, h // rep])
        want = p / l @ vv
        spread = p / l @ np.abs(vv)
        b = spread * (lu.BF16 + (160 + 16 + n + 8) * 2.0 ** -23)
        bound = b + lu.BF16 * (np.abs(want) + b)
        # (a result of zeros, or of one key more or less, does not meet it)
        assert (bound < 0.02 * np.abs(want)).all()
        lu.check(lu.f64(got[:, h]), want, bound, "head %d" % h)
        ll = (top + np.log(l))[:, 0]
        lu.check(lu.f64(lse[:, h]), ll, np.abs(ll) * 2.0 ** -22 + (n + 200) * 2.0 ** -23, "lse %d" % h)


def numbers(m, n, d, seed, base):
    """Scores base[j] + a whole number from 0 to 9 that depends on query and key; values from 1 to 3."""
    q = torch.zeros((m, 4, d), device="cuda")
    q[..., 0], q[..., d - 1] = 1.0, 1.0
    q[..., 1:9] = (rand((m, 4, 8), seed) < 0.5).float()
    k = torch.zeros((n, 2, d), device="cuda")
    k[..., 0] = base[:, None]
    k[..., 1:9] = (rand((n, 2, 8), seed + 1) < 0.4).float()
    k[..., d - 1] = (rand((n, 2), seed + 2) < 0.3).float()
    v = 1.0 + 2.0 * rand((n, 2, d), seed + 3)
    return q.bfloat16(), k.bfloat16(), v.bfloat16()


def bases(n):
    """What all of a key's scores have in common, named: 2^20 and more is where exponents are formed
    from differences of scores."""
    j = torch.arange(n, device="cuda")
    far = lambda on: torch.where(on, 2.0 ** 20, 0.0)
    return {
        "none": far(j < 0),
        "large": far(j >= 0),
        "large below zero": -far(j >= 0),
        "larger": 8 * far(j >= 0),
        "large from the middle of the whole steps on": far(j >= n * 5 // 8 + 7),
        "large at the end": far(j >= n - 40),
        "large below zero, then none": -far(j < n // 2 + 11),
        "one large key": far(j == n // 3),
        "large and larger in turn": far(j >= 0) * (1 + (j // 100) % 4),
        "up": 2.0 ** 14 * (j // 64),
    }


NAMES = ["none", "large", "large below zero", "larger", "large from the middle of the whole steps on",
         "large at the end", "large below zero, then none", "one large key", "large and larger in turn", "up"]


@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("name", NAMES)
def test_scores_far_from_zero(d, name):
    n = 900
    q, k, v = numbers(n, n, d, 11, bases(n)[name])
    out, lse = fq.prompt_attention(q, k, v, offsets(n), scale=1.0, lse=True)
    exact(q, k, v, out, lse)
    # the other sign of both
    out, lse = fq.prompt_attention(-q, k, v, offsets(n), scale=-1.0, lse=True)
    exact(q, k, v, out, lse)


@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("name", NAMES)
def test_scores_far_from_zero_in_parts(d, name):
    m, n = 21, 3500
    q, k, v = numbers(m, n, d, 13, bases(n)[name])
    assert fq.rollout_lib().prompt_attention_workspace_bytes(m, 4, n, 2, d, 1) > 0
    out, lse = fq.prompt_attention(q, k, v, offsets(m), offsets(n), scale=1.0, lse=True)
    exact(q, k, v, out, lse)


def test_offsets_past_the_ends_leave_other_sequences_right():
    q, k, v = numbers(64, 64, 64, 17, bases(64)["none"])
    as_offsets = lambda o: torch.tensor(o, dtype=torch.int32, device="cuda")
    # queries and keys of each sequence as the clamped offsets give them
    for q_off, k_off, spans in (
            ([-5, 20, 900], [0, 20, 2000], [(0, 20, 0, 20), (20, 64, 20, 64)]),
            ([0, 30, 64], [-9, 30, 5000], [(0, 30, 0, 30), (30, 64, 30, 64)]),
            ([0, 64, 10], [0, 64, 64], [(0, 64, 0, 64)]),
            ([0, 10, 70], [0, 30, 90], [(0, 10, 0, 30), (10, 64, 30, 64)])):
        out, lse = fq.prompt_attention(q, k, v, as_offsets(q_off), as_offsets(k_off), scale=1.0, lse=True)
        for a, b, c, e in spans:
            if b - a > e - c:  # the first queries see nothing
                empty = b - a - (e - c)
                assert (out[a:a + empty] == 0).all() and (lse[a:a + empty] == -math.inf).all()
                a += empty
            exact(q[a:b], k[c:e], v[c:e], out[a:b], lse[a:b])
    # past both ends: no row is any sequence's
    out = torch.full_like(q, 7.0)
    fq.prompt_attention(q, k, v, as_offsets([70, 80, 90]), as_offsets([70, 80, 90]), out=out)
    assert (out == 7).all()
