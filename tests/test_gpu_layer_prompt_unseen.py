"""prompt_attention: what a query does not see changes no bit of its result, at
every step of its keys, in wholes and in parts."""
import math

import numpy as np
import pytest
import torch

import fp4_block_quantization_amd as fq

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


def rising(m, n, d, seed, slope=0.025):
    """Queries and keys whose scores (with a scale of 1) rise slowly, by less than the running
    maximum's slack from any step to the last, so that only the first step moves it."""
    q = torch.zeros((m, 4, d), device="cuda")
    q[..., 0], q[..., 1:] = 1.0, 0.02 * (rand((m, 4, d - 1), seed) - 0.5)
    k = torch.zeros((n, 2, d), device="cuda")
    k[..., 0] = slope * (torch.arange(n, device="cuda") - (n - 200)).clamp(min=0)[:, None]
    k[..., 1:] = rand((n, 2, d - 1), seed + 1) - 0.5
    v = 2.0 * rand((n, 2, d), seed + 2) - 1.0
    return q.bfloat16(), k.bfloat16(), v.bfloat16()


# a key that the last queries see and the others do not: what it is worth
KEYS = [40.0, 2.0 ** 22, -2.0 ** 22, math.inf, -math.inf, math.nan]


@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("at", [5, 70, 135, 190])
def test_a_key_that_a_query_does_not_see_changes_no_bit(d, at):
    q, k, v = rising(200, 200, d, 1)
    clean, lse = fq.prompt_attention(q, k, v, offsets(200), scale=1.0, lse=True)
    for worth in KEYS:
        kk = k.clone()
        kk[at, 1, 0] = worth
        out, l = fq.prompt_attention(q, kk, v, offsets(200), scale=1.0, lse=True)
        assert torch.equal(out[:at], clean[:at]), worth
        assert torch.equal(l[:at], lse[:at]), worth
        assert torch.equal(out[:, :2], clean[:, :2]) and torch.equal(l[:, :2], lse[:, :2])
        if worth in (40.0, 2.0 ** 22):  # it has all the weight, but for e^-30
            assert torch.equal(out[at:, 2:], v[at, 1].expand(200 - at, 2, d))
        elif not math.isfinite(worth) and worth != -math.inf:
            assert torch.isnan(out[at:, 2:]).all()
        else:
            assert torch.isfinite(out).all()


@pytest.mark.parametrize("d", DIMS)
def test_a_key_that_a_query_does_not_see_changes_no_bit_of_parts(d):
    # ten queries behind a long context that is cut into parts
    q, k, v = rising(10, 4000, d, 3)
    off = offsets(10), offsets(4000)
    assert fq.rollout_lib().prompt_attention_workspace_bytes(10, 4, 4000, 2, d, 1) > 0
    clean, lse = fq.prompt_attention(q, k, v, *off, scale=1.0, lse=True)
    for worth in KEYS:
        kk = k.clone()
        kk[3995, 1, 0] = worth  # seen by the last five
        out, l = fq.prompt_attention(q, kk, v, *off, scale=1.0, lse=True)
        assert torch.equal(out[:5], clean[:5]) and torch.equal(l[:5], lse[:5]), worth
        assert torch.equal(out[:, :2], clean[:, :2])


@pytest.mark.parametrize("d", DIMS)
def test_a_long_prompts_unseen_keys(d):
    # many whole steps before: the inner loop is left, and come back to, at other steps
    n, at = 1500, 1400
    q, k, v = rising(n, n, d, 5)
    clean, lse = fq.prompt_attention(q, k, v, offsets(n), scale=1.0, lse=True)
    for worth in KEYS:
        kk = k.clone()
        kk[at, 1, 0] = worth
        out, l = fq.prompt_attention(q, kk, v, offsets(n), scale=1.0, lse=True)
        assert torch.equal(out[:at], clean[:at]) and torch.equal(l[:at], lse[:at]), worth
