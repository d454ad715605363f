"""prompt_attention's weights add up to one: where all values of a sequence are
alike, they are its result to the bit, whatever the scores."""
import numpy as np
import pytest
import torch

import fp4_block_quantization_amd as fq
import layerutil as lu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.rollout_lib()


def inputs(q_lens, k_lens, d, gain):
    g = torch.Generator(device="cuda").manual_seed(d + sum(k_lens))
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    q, k = gain * rnd(sum(q_lens), 4, d), rnd(sum(k_lens), 2, d)
    one = rnd(len(k_lens), 2, d)  # a sequence's and key head's value
    v = one.repeat_interleave(torch.tensor(k_lens, device="cuda"), 0)
    want = one.repeat_interleave(torch.tensor(q_lens, device="cuda"), 0).repeat_interleave(2, 1)
    return q.bfloat16(), k.bfloat16(), v.bfloat16(), want.bfloat16()


def offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("gain", [0.0, 0.3, 1.0, 6.0])
@pytest.mark.parametrize("q_lens,k_lens", [([1, 2, 3, 70, 129, 200], [1, 2, 3, 70, 129, 200]), ([700], [700]),
                                           ([3, 70], [300, 900]), ([9], [4000]), ([2, 30], [3000, 1500])])
def test_equal_values(d, gain, q_lens, k_lens):
    # (the sums are off by (keys + 8) 2^-23 at most, and a value is a BF16 number: nothing within
    # 2^-9 of it rounds to another)
    q, k, v, want = inputs(q_lens, k_lens, d, gain)
    out = fq.prompt_attention(q, k, v, offsets(q_lens), offsets(k_lens))
    assert torch.equal(out, want)
    again, lse = fq.prompt_attention(q, k, v, offsets(q_lens), offsets(k_lens), lse=True)
    assert torch.equal(again, want)
    # the log-sum-exp takes the probabilities before they are rounded
    a = c = 0
    for m, n in zip(q_lens, k_lens):
        kk, vv = (np.repeat(lu.f64(t[c:c + n]), 2, 1) for t in (k, v))
        _, l, _, bound = lu.prompt(lu.f64(q[a:a + m]), kk, vv, d ** -0.5)
        lu.check(lu.f64(lse[a:a + m]), l, bound, "lse of %d of %d" % (m, n))
        a, c = a + m, c + n
