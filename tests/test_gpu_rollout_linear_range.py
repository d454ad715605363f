"""nvfp4_linear and mxfp4_linear at the ends of their inputs' range, in every
form: an infinite activation in a row's last elements, and every E8M0 byte."""
import numpy as np
import pytest
import torch

import fp4_block_quantization_amd as fq
import rolloututil as ru
import workloads
from gpuutil import to_dev

pytestmark = pytest.mark.gpu

ROWS = [1, 2, 3, 16, 20, 70]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.rollout_lib()


def product_bound(x, w):
    """y = x . w^T in float64 and the bound of FP32 sums: k additions, each off by at most 2^-23
    of the sum of magnitudes, the scale products, and FP32's subnormals."""
    mag = np.abs(x) @ np.abs(w).T
    return x @ w.T, (x.shape[1] + 8) * 2.0 ** -23 * mag + 2.0 ** -140


def run(mx, x_bits, q, grouped):
    x = to_dev(x_bits)
    q = [torch.from_numpy(a).cuda() for a in q]
    offsets = None
    if grouped:  # the matrix as the second of two experts
        q = [torch.stack([torch.zeros_like(a), a]) for a in q]
        offsets = torch.tensor([0, 0, x.shape[0]], device="cuda")
    call = fq.mxfp4_linear if mx else fq.nvfp4_linear
    return call(x, *q, offsets=offsets, out_dtype=torch.float32).cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("mx,k", [(False, 16), (False, 48), (False, 80), (False, 528), (False, 2064),
                                  (False, 7152), (True, 32), (True, 96), (True, 544), (True, 2080),
                                  (True, 7200)])
def test_an_infinity_in_the_last_elements(mx, k, rows, grouped):
    # no weight is zero, so the product is infinite with the weight's sign
    n = 37
    rng = np.random.default_rng(k + rows)
    codes = rng.choice([c for c in range(256) if c % 8 and c // 16 % 8], (n, k // 2)).astype(np.uint8)
    if mx:
        q = (codes, np.full((n, k // 32), 125, np.uint8))
        w = ru.mx_values(*q)
    else:
        q = (codes, np.full((n, k // 16), 0x33, np.uint8), np.full(n, 0.5, np.float32))
        w = ru.nv_values(*q)
    x = workloads.random_rows(rows, rows, k)
    finite = run(mx, x, q, grouped)
    want, bound = product_bound(ru.bf16_values(x), w)
    ru.check(finite, want, bound, "finite")
    for at in (k - 1, k - 8, k - 9):
        for row in {0, rows - 1}:
            y = x.copy()
            y[row, at] = 0x7F80
            got = run(mx, y, q, grouped)
            assert np.array_equal(got[row], np.where(w[:, at] < 0, -np.inf, np.inf)), (at, row)
            keep = np.arange(rows) != row
            assert np.array_equal(got[keep], finite[keep])


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("k", [32, 96, 544, 4128])
def test_every_scale_byte(k, rows, grouped):
    # one byte a column: weights from 2^-128 (subnormal numbers of BF16) to 6 * 2^128, which
    # neither BF16 nor FP32 holds; products with activations that bring them into FP32's range
    codes = np.random.default_rng(k + rows).integers(0, 256, (256, k // 2)).astype(np.uint8)
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], k // 32, 1)
    w = ru.mx_values(codes, scales)
    base = ru.bf16_values(workloads.random_rows(rows, rows, k))
    for power, cols in ((100, slice(0, 100)), (0, slice(20, 230)), (-60, slice(90, 256))):
        x = workloads.to_bf16_bits((base * 2.0 ** power).astype(np.float32))
        got = run(True, x, (codes[cols], scales[cols]), grouped)
        want, bound = product_bound(ru.bf16_values(x), w[cols])
        ru.check(got, want, bound, "2^%d" % power)


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("rows", ROWS)
def test_scale_bytes_of_a_column_far_apart(rows, grouped):
    # neighbouring blocks from the lowest byte to the highest, met by activations to match
    n, k = 48, 1056
    rng = np.random.default_rng(rows)
    codes = rng.integers(0, 256, (n, k // 2)).astype(np.uint8)
    byte = rng.permutation(np.linspace(0, 255, k // 32).astype(np.int64))
    scales = np.repeat(byte[None].astype(np.uint8), n, 0)
    x = ru.bf16_values(workloads.random_rows(rows, rows, k))
    x *= 2.0 ** np.repeat(np.clip(127 - byte, -110, 110), 32)[None]
    x = workloads.to_bf16_bits(x.astype(np.float32))
    got = run(True, x, (codes, scales), grouped)
    want, bound = product_bound(ru.bf16_values(x), ru.mx_values(codes, scales))
    ru.check(got, want, bound, "far apart")
