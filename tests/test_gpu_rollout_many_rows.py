"""nvfp4_kv_attention with more workgroups, and more query rows, than one
launch takes: queries are repetitions of a few, so that outputs must repeat
too, and a few of them are checked against a small call's."""
import numpy as np
import pytest
import torch

import fp4_block_quantization_amd as fq
import workloads
from gpuutil import to_dev

pytestmark = pytest.mark.gpu
DIM, PAGE = 64, 16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.rollout_lib()
    yield
    torch.cuda.empty_cache()


def filled(pages, heads):
    cache = fq.nvfp4_kv_cache(pages, PAGE, heads, DIM)
    k, v = (to_dev(workloads.random_rows(s, pages * PAGE * heads, DIM)).view(-1, heads, DIM)
            for s in (1, 2))
    fq.nvfp4_kv_append(cache, k, v, torch.arange(pages * PAGE, device="cuda"))
    return cache


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def near(got, want):
    """Two roundings to BF16, and FP16 probabilities."""
    got, want = got.float(), want.float()
    assert ((got - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -9 * want.abs().max()).all()


@pytest.mark.parametrize("grouped", [False, True])
def test_more_workgroups_than_one_launch_takes(grouped):
    # one token of 65535 sequences, 72 heads of their own cache head each: 4.7e6 items
    batch, heads, period = 65535, 72, 257
    cache = filled(4, heads)
    q = to_dev(workloads.random_rows(3, period * heads, DIM)).view(period, heads, DIM)
    times = -(-batch // period)
    lens = torch.arange(period, dtype=torch.int32, device="cuda") % (2 * PAGE + 1)
    table = i32(2, 0).repeat(period, 1)
    prefix = lambda n: (i32(3, 1)[None], i32(27), i32(0, n)) if grouped else None
    small = fq.nvfp4_kv_attention(q, cache, table, lens, prefix=prefix(period))
    big, lse = fq.nvfp4_kv_attention(
        q.repeat(times, 1, 1)[:batch], cache, table.repeat(times, 1)[:batch],
        lens.repeat(times)[:batch], prefix=prefix(batch), lse=True)
    assert torch.isfinite(lse if grouped else lse[1]).all()
    first = big[:period]
    near(first, small)
    for i in range(0, batch, period):
        n = min(period, batch - i)
        if grouped:  # a block of 16 rows of the prefix joins other sequences each time
            near(big[i:i + n], small[:n])
        else:
            assert torch.equal(big[i:i + n], first[:n]), i


@pytest.mark.parametrize("grouped", [False, True])
def test_more_rows_than_one_launch_takes(grouped):
    # two sequences of 4.4e6 queries, of which all but the last see the prefix alone, or nothing
    batch, tokens, period, own = 2, 4400001, 4096, 30
    cache = filled(8, 1)
    q = to_dev(workloads.random_rows(5, period, DIM)).view(period, 1, DIM)
    q = q.repeat(-(-tokens // period), 1, 1)[:tokens]
    q = torch.stack([q, q.flip(0)])
    table, lens = i32(2, 0, 5, 1)[None].repeat(2, 1)[:, :2].contiguous(), i32(own, own - 7)
    prefix = lambda n: (i32(3, 4, 6)[None], i32(41), i32(0, n)) if grouped else None
    big, lse = fq.nvfp4_kv_attention(q, cache, table, lens, prefix=prefix(batch), lse=True)
    last = 64
    small = fq.nvfp4_kv_attention(q[:, -last:].contiguous(), cache, table, lens,
                                  prefix=prefix(batch))
    near(big[:, -last:], small)
    if not grouped:
        assert not big[:, :tokens - own].any()
        assert torch.isneginf(lse[:, :tokens - own]).all()
        return
    seen = fq.nvfp4_kv_attention(q[:1, :period].contiguous(), cache, table[:1], i32(0),
                                 prefix=prefix(1))[0]
    for i in range(0, tokens - own - period, period):
        near(big[0, i:i + period], seen)
        near(big[1, tokens - i - period:tokens - i].flip(0)[own:], seen[own:])
