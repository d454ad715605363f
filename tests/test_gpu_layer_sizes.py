"""Sizes that the layer operators refuse are refused before memory is asked for."""
import pytest
import torch

import fp4_block_quantization_amd as fq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.rollout_lib()


def test_sizes_are_refused_before_memory_is_asked_for():
    logits = torch.randn((6, 16), device="cuda")
    x, e = torch.randn((6, 32), device="cuda").bfloat16(), torch.zeros((6, 2), dtype=torch.int32, device="cuda")
    for big in (1 << 40, 1 << 62, (1 << 63) - 1):
        with pytest.raises(fq.Fp4qError):
            fq.moe_route(logits, big)
        with pytest.raises(fq.Fp4qError):
            fq.moe_dispatch(x, e, big)
    before = torch.cuda.memory_allocated()
    for call in (lambda: fq.moe_route(logits, 65), lambda: fq.moe_dispatch(x, e, 1025)):
        with pytest.raises(fq.Fp4qError):
            call()
    assert torch.cuda.memory_allocated() == before
