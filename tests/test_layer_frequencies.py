"""rotary_frequencies refuses what does not give finite frequencies."""
import math

import pytest

import fp4_block_quantization_amd as fq


def test_frequencies_that_are_not_finite_are_refused():
    for kw in (dict(dims=4, method="base", factor=1e200), dict(dims=64, base=1e-320),
               dict(dims=64, method="positions", factor=1e-320, base=1e-300),
               dict(dims=8, method="parts", factor=2.0, original_positions=math.nan),
               dict(dims=8, method="parts", factor=2.0, original_positions=100, slow=-math.inf, fast=math.inf)):
        with pytest.raises(fq.Fp4qError):
            fq.rotary_frequencies(device="cpu", **kw)


def test_large_and_small_ones_are_taken():
    for kw in (dict(dims=64, base=1e300), dict(dims=64, base=1e-5), dict(dims=64, method="positions", factor=1e300),
               dict(dims=8, method="parts", factor=2.0, original_positions=math.inf),
               dict(dims=8, method="parts", factor=2.0, original_positions=100, fast=math.inf)):
        f, a = fq.rotary_frequencies(device="cpu", **kw)
        assert f.isfinite().all() and math.isfinite(a)
