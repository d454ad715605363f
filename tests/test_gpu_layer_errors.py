"""The layer operators report their own errors, and no other call's."""
import pytest
import torch

import fp4_block_quantization_amd as fq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.rollout_lib()


def test_an_error_left_by_another_call_is_not_this_ones():
    tokens, k = 5000, 2  # in several launches
    x = torch.randn((tokens, 16), device="cuda").bfloat16()
    w, e = fq.moe_route(torch.randn((tokens, 8), device="cuda"), k)
    rows, off, place = fq.moe_dispatch(x, e, 8)
    want = fq.moe_combine(rows, place, w)
    ws = torch.empty(fq.rollout_lib().moe_dispatch_workspace_bytes(tokens, k, 8), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(rows), torch.empty_like(off), torch.empty_like(place)
    back = torch.empty_like(x)
    torch.cuda.synchronize()
    runtime = fq.rollout_lib()  # (the runtime's calls are found through the library that uses it)
    try:
        assert runtime.hipSetDevice(10000) != 0  # refused by the runtime, which remembers it
        fq.moe_dispatch(x, e, 8, out=out, workspace=ws)
        assert runtime.hipSetDevice(10000) != 0
        fq.moe_combine(rows, place, w, out=back)
    finally:
        runtime.hipGetLastError()
    assert torch.equal(out[2], place) and torch.equal(back, want)
