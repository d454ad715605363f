"""rotary at positions so far that their angles are known only from the exact
product: against sines and cosines of angles reduced in whole numbers."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import fp4_block_quantization_amd as fq
import layerutil as lu

pytestmark = pytest.mark.gpu

BITS = 400


def arctan_of_inverse(n):
    """2^BITS arctan(1 / n), off by a few units."""
    total, power, i = 0, (1 << BITS) // n, 0
    while power:
        total += power // (2 * i + 1) * (-1) ** i
        power //= n * n
        i += 1
    return total


# pi / 4 = 4 arctan(1/5) - arctan(1/239)
TURN = Fraction(8 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239)), 1 << BITS)


def rest_of(position, frequency):
    """The angle less whole turns, exactly but for 2^-300 of it."""
    angle = Fraction(position) * Fraction(frequency)
    return float(angle - TURN * round(angle / TURN))


def test_the_reduction():
    assert abs(float(TURN) - 2 * math.pi) < 1e-15
    for p, f in ((3, 1.0), (100, 0.25), (-7, 1.5), (12345, 1e-4)):
        assert abs(math.sin(rest_of(p, f)) - math.sin(p * f)) < 1e-11


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.rollout_lib()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("start", [0, 1 << 27, 1 << 30, 1 << 40, (1 << 50) + 12345, (1 << 53) - 40, -(1 << 45), 5 - (1 << 53)])
def test_far_positions(start, dtype, interleaved):
    tokens, d = 33, 64
    f, amplitude = fq.rotary_frequencies(d, method="parts", factor=4.0, original_positions=4096)
    f[1], f[2], f[3] = math.pi / 2, 3.0, 1e-9
    pos = start + torch.arange(tokens, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn((tokens, 3, d), generator=g, device="cuda").to(dtype)
    rest = np.array([[rest_of(int(p), float(w)) for w in f.tolist()] for p in pos.tolist()])[:, None]
    a, b = (slice(0, d, 2), slice(1, d, 2)) if interleaved else (slice(0, d // 2), slice(d // 2, d))
    for inverse in (False, True):
        got = lu.f64(fq.rotary(x, None, pos, f, amplitude=amplitude, interleaved=interleaved, inverse=inverse)[0])
        xx = lu.f64(x)
        c, s = np.cos(rest) * amplitude, np.sin(rest) * amplitude * (-1 if inverse else 1)
        want = np.zeros_like(xx)
        want[..., a], want[..., b] = xx[..., a] * c - xx[..., b] * s, xx[..., b] * c + xx[..., a] * s
        # sine and cosine within 2^-23, their products with the amplitude, the two products and
        # their sum round (FP32), then the result
        off = np.zeros_like(xx)
        off[..., a] = off[..., b] = (np.abs(xx[..., a]) + np.abs(xx[..., b])) * amplitude * (2.0 ** -23 + 4 * lu.FP32)
        if dtype is torch.bfloat16:
            off = off + lu.BF16 * (np.abs(want) + off)
        lu.check(got, want, off + 1e-44, "from %d" % start)


def test_angles_past_2_to_the_53rd():
    # (frequencies of any size are taken: 2^60 radians and more)
    pos = torch.tensor([(1 << 53) - 1, 3, -(1 << 52) - 1, 1 << 40, 12345678901], device="cuda")
    f = torch.tensor([1000.5, 2.0 ** 10 + 2.0 ** -40, 1e6 / 3, 7.0], dtype=torch.float64, device="cuda")
    x = torch.randn((5, 2, 8), device="cuda")
    rest = np.array([[rest_of(int(p), float(w)) for w in f.tolist()] for p in pos.tolist()])[:, None]
    xx, c, s = lu.f64(x), np.cos(rest), np.sin(rest)
    want = np.concatenate([xx[..., :4] * c - xx[..., 4:] * s, xx[..., 4:] * c + xx[..., :4] * s], -1)
    off = np.tile((np.abs(xx[..., :4]) + np.abs(xx[..., 4:])) * (2.0 ** -23 + 4 * lu.FP32), 2)
    lu.check(lu.f64(fq.rotary(x, None, pos, f)[0]), want, off, "past 2^53")
