"""nvfp4_kv_attention over contexts of many parts, against float64: the join
of partial results takes four further parts at a time on each of LANES groups
of threads (one row a workgroup) or on one (several rows), so an item's count
of further parts goes through several such rounds here, with a last round
that is full, and one of a single part."""
import numpy as np
import pytest
import torch

import fp4_block_quantization_amd as fq
from gpuutil import bits_of
from test_gpu_rollout_attention import Batch

pytestmark = pytest.mark.gpu

PART = 512  # tokens of the shortest part
LANES = {64: 16, 128: 8, 192: 5, 256: 4}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.rollout_lib()


def check_repeats(b):
    """Equal bit for bit, call after call, on whatever the workspace holds."""
    first = b.run(lse=True)
    for fill in (0, 0xFF):
        ws = torch.full((1 << 26,), fill, dtype=torch.uint8, device="cuda")
        again = b.run(lse=True, workspace=ws)
        assert np.array_equal(bits_of(first[0]), bits_of(again[0]))
        assert torch.equal(first[1], again[1])


@pytest.mark.parametrize("more", [0, 1])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_one_long_context(dim, more):
    # 8 LANES further parts, and one more
    tokens = PART * (8 * LANES[dim] + 1) + more
    b = Batch(dim + more, [tokens], heads=3, kv_heads=1, dim=dim, page=64)
    b.check(label="%d tokens" % tokens)
    check_repeats(b)


@pytest.mark.parametrize("parts", [13, 14])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_one_long_context_among_many_rows(dim, parts):
    lens = [i % 23 for i in range(130)]
    lens[77] = PART * parts - 5
    b = Batch(parts + dim, lens, heads=8, kv_heads=1, dim=dim, page=128)
    b.check(label="%d parts" % parts)
    check_repeats(b)


@pytest.mark.parametrize("more", [0, 1])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_a_long_prefix(dim, more):
    tokens = PART * (8 * LANES[dim] + 1) + more
    b = Batch(5 + dim, [3, 0, 70], heads=2, kv_heads=1, dim=dim, page=64, prefix_lens=[tokens],
              members=[0, 2])
    b.check(label="prefix of %d" % tokens)
    check_repeats(b)


@pytest.mark.parametrize("tiles", [200, 209])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_long_prefix_of_many_rows(dim, tiles):
    # 1040 rows: 33 blocks of 32 (heads up to 128) or 65 of 16, and 512 parts in all, so about
    # 13 and 14, or 7, parts a block
    b = Batch(tiles + dim, [i % 5 for i in range(130)], heads=8, kv_heads=1, dim=dim, page=64,
              prefix_lens=[64 * tiles], members=[0, 130])
    b.check(label="prefix of %d tiles" % tiles)
    check_repeats(b)
