"""Outputs of one call of the layer operators stay apart, whatever is done with
one of them."""
import pytest
import torch

import fp4_block_quantization_amd as fq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.rollout_lib()


def outputs(tokens):
    f, _ = fq.rotary_frequencies(64)
    x = torch.randn((tokens, 6, 64), device="cuda").bfloat16()
    yield fq.rotary(x[:, :4], x[:, 4:], torch.arange(tokens, device="cuda"), f)
    yield fq.prompt_attention(x[:, :4], x[:, 4:5], x[:, 5:], torch.tensor([0, tokens], device="cuda").int(), lse=True)
    w, e = fq.moe_route(torch.randn((tokens, 9), device="cuda"), 3)
    chosen = e.clone()  # (what is yielded gets resized)
    yield w, e
    yield fq.moe_dispatch(x.view(tokens, 384), chosen, 9)


@pytest.mark.parametrize("tokens", [1, 7, 300])
@pytest.mark.parametrize("how", ["resize", "out", "fill"])
@pytest.mark.filterwarnings("ignore:An output with one or more elements was resized")
def test_an_output_that_grows_leaves_the_others(tokens, how):
    for outs in outputs(tokens):
        assert all(t.is_contiguous() and not t.requires_grad and not t._is_view() for t in outs)
        assert all(t.data_ptr() % 16 == 0 for t in outs)
        for i, t in enumerate(outs):
            kept = [o.clone() for o in outs]
            if how == "resize":
                t.resize_(3 * t.numel() + 100).fill_(7)
            elif how == "out":
                torch.add(torch.full((3 * t.numel() + 100,), 7, dtype=t.dtype, device="cuda"), 0, out=t)
            else:
                t.fill_(7)
            assert (t == 7).all()
            for j, o in enumerate(outs):
                assert j <= i or torch.equal(o, kept[j]), (i, j)


def test_outputs_keep_their_own_memory_alone():
    for outs in outputs(50):
        for t in outs:
            assert t.storage_offset() == 0
            assert t.untyped_storage().nbytes() == t.numel() * t.element_size()
