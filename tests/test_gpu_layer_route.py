"""moe_route against float64: experts equal, weights within their bounds; ties,
groups, biases, infinities and NaN, padding."""
import math

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


def logits_of(tokens, experts, dtype, seed=0, gain=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed + tokens + 31 * experts)
    return (gain * torch.randn((tokens, experts), generator=g, device="cuda")).to(dtype)


def check(logits, got, top_k, bias=None, scoring="softmax", groups=1, top_groups=1, renormalize=True,
          scale=1.0, label=""):
    x = lu.f64(logits)
    w, e = lu.route(x, top_k, None if bias is None else lu.f64(bias), scoring, groups, top_groups,
                    renormalize, scale)
    assert got[1].dtype is torch.int32 and got[0].dtype is torch.float32
    assert np.array_equal(got[1].cpu().numpy(), e), label
    # each exponential: its argument rounds (FP32: 2^-24 of it), the function to 2 units; the sum
    # of up to all experts' (2^-24 for each addition); the quotients and the scale
    spread = (np.abs(x).max(1) * 2)[:, None]
    rel = (spread + 16 + x.shape[1]) * 2.0 ** -23
    lu.check(got[0].cpu().numpy(), w, np.abs(w) * rel + 1e-37, label)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("experts,top_k", [(1, 1), (2, 1), (7, 7), (64, 8), (65, 3), (128, 8), (200, 64), (256, 6),
                                           (511, 5), (1024, 10)])
def test_experts(experts, top_k, renormalize, scoring, dtype):
    for tokens in (1, 6, 37):
        x = logits_of(tokens, experts, dtype)
        got = fq.moe_route(x, top_k, scoring=scoring, renormalize=renormalize, scale=2.5)
        check(x, got, top_k, None, scoring, renormalize=renormalize, scale=2.5, label="%d tokens" % tokens)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("experts,groups,top_groups,top_k", [
    (256, 8, 4, 8), (64, 64, 3, 3), (64, 64, 64, 64), (6, 2, 1, 3), (96, 3, 2, 5), (1024, 2, 1, 8), (10, 5, 5, 4),
    (512, 16, 1, 6), (35, 7, 2, 1), (33, 33, 8, 8)])
def test_groups(experts, groups, top_groups, top_k, with_bias, scoring, dtype):
    x = logits_of(29, experts, dtype)
    bias = 0.1 * torch.randn(experts, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)) \
        if with_bias else None
    got = fq.moe_route(x, top_k, bias=bias, scoring=scoring, groups=groups, top_groups=top_groups)
    check(x, got, top_k, bias, scoring, groups, top_groups, label="groups")


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_index(scoring):
    x = torch.zeros((3, 130), device="cuda")
    x[1, 70:] = 1.0
    x[2, [5, 69, 129]] = 2.0
    x[2, 6] = -0.0
    for bias in (None, torch.zeros(130, device="cuda")):
        w, e = fq.moe_route(x, 5, bias=bias, scoring=scoring)
        assert e.tolist() == [[0, 1, 2, 3, 4], [70, 71, 72, 73, 74], [5, 69, 129, 0, 1]]
    _, e = fq.moe_route(torch.zeros((1, 64), device="cuda"), 9, scoring=scoring, groups=8, top_groups=2)
    assert e.tolist() == [list(range(9))]


def test_keys_that_fp32_does_not_tell_apart():
    # scores that differ by 2^-30 of them; the bias moves them into the order of the scores
    x = torch.zeros((1, 64), device="cuda")
    x[0, 20], x[0, 40] = 2.0 ** -28, 2.0 ** -27
    w, e = fq.moe_route(x, 3, bias=torch.full((64,), 0.25, device="cuda"), scoring="sigmoid")
    assert e.tolist() == [[40, 20, 0]]
    # and against a bias that differs by less than an FP32 sum keeps
    bias = torch.full((64,), 64.0, device="cuda")
    x = torch.zeros((1, 64), device="cuda")
    x[0, 33] = 2.0 ** -20
    _, e = fq.moe_route(x, 2, bias=bias, scoring="sigmoid")
    assert e.tolist() == [[33, 0]]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_infinities(scoring, with_bias):
    # experts that are shut off: never chosen before others, without weight
    x = logits_of(20, 40, torch.float32)
    x[:, 3::4] = -math.inf
    x[5] = -math.inf
    x[6, 1:] = -math.inf
    bias = torch.linspace(0, 0.1, 40, device="cuda") if with_bias else None
    for renormalize in (False, True):
        w, e = fq.moe_route(x, 6, bias=bias, scoring=scoring, renormalize=renormalize)
        ww, ee = lu.route(lu.f64(x), 6, None if bias is None else lu.f64(bias), scoring, 1, 1, renormalize, 1.0)
        assert np.array_equal(e.cpu().numpy(), ee)
        assert np.allclose(w.cpu().numpy(), ww, rtol=1e-4, atol=1e-37)
    assert (w[5] == 0).all() and w[6, 0 if not with_bias else e[6].tolist().index(0) if 0 in e[6].tolist() else 0] >= 0


def test_nan_logits_keep_the_choice_in_range():
    for experts, groups in ((8, 1), (64, 8), (300, 1)):
        for bias in (None, torch.zeros(experts, device="cuda")):
            for scoring in ("softmax", "sigmoid"):
                x = logits_of(12, experts, torch.float32)
                x[0], x[1, 2], x[2, ::2], x[3, 1:] = math.nan, math.nan, math.nan, math.nan
                x[4], x[5, 3] = math.inf, math.inf
                w, e = fq.moe_route(x, 4, bias=bias, scoring=scoring, groups=groups, top_groups=groups)
                assert ((e >= 0) & (e < experts)).all()
                assert all(len(set(r)) == 4 for r in e.tolist())
                clean = fq.moe_route(x[6:].contiguous(), 4, bias=bias, scoring=scoring, groups=groups,
                                     top_groups=groups)
                assert torch.equal(w[6:], clean[0]) and torch.equal(e[6:], clean[1])
                if bias is None and groups == 1:  # behind every other
                    assert 2 not in e[1].tolist() and e[3, 0] == 0


def test_inactive_tokens_and_out():
    x = logits_of(50, 32, torch.bfloat16)
    active = torch.arange(50, device="cuda") % 3 != 1
    want = fq.moe_route(x, 4)
    out = (torch.full((50, 4), 9.0, device="cuda"), torch.full((50, 4), 9, dtype=torch.int32, device="cuda"))
    got = fq.moe_route(x, 4, active=active, out=out)
    assert got[0].data_ptr() == out[0].data_ptr() and got[1].data_ptr() == out[1].data_ptr()
    assert torch.equal(got[0][active], want[0][active]) and torch.equal(got[1][active], want[1][active])
    assert (got[0][~active] == 0).all() and (got[1][~active] == -1).all()
    assert fq.moe_route(x[:0], 4)[0].shape == (0, 4)


def test_weights_that_underflow():
    x = torch.tensor([[-200.0, -150.0, -300.0, -1000.0], [300.0, -300.0, 200.0, 0.0]], device="cuda")
    w, e = fq.moe_route(x, 2, scoring="sigmoid")
    assert e.tolist() == [[1, 0], [0, 2]] and (w[0] == 0).all() and w[1].tolist() == [0.5, 0.5]
    w, e = fq.moe_route(x, 2, renormalize=False)
    # (e^-100 is 26.5 of FP32's smallest steps, 2^-149, and no zero)
    assert e.tolist() == [[1, 0], [0, 2]] and w[1, 0] == 1.0
    assert abs(w[1, 1].item() - math.exp(-100)) <= 2.0 ** -149
    # relative to the largest chosen, not to the largest of all
    bias = torch.tensor([0.0, 0.0, 5.0, 6.0], device="cuda")
    w, e = fq.moe_route(torch.tensor([[0.0, 0.0, -200.0, -200.0]], device="cuda"), 2, bias=bias)
    assert e.tolist() == [[3, 2]] and w.tolist() == [[0.5, 0.5]]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,top_groups,top_k", [
    (64, 1, 1, 9), (100, 1, 1, 64), (256, 1, 1, 10), (256, 8, 3, 33), (512, 1, 1, 64), (1024, 1, 1, 40),
    (1024, 16, 5, 20)])
def test_many_equal_keys_with_a_bias(experts, groups, top_groups, top_k, scoring):
    # two logits and two biases: a few keys, many experts of each, in one lane and in several
    g = torch.Generator(device="cuda").manual_seed(experts + groups)
    x = torch.randint(0, 2, (21, experts), generator=g, device="cuda").float()
    x[:3] = 0.5
    bias = torch.randint(0, 2, (experts,), generator=g, device="cuda").float()
    got = fq.moe_route(x, top_k, bias=bias, scoring=scoring, groups=groups, top_groups=top_groups)
    check(x, got, top_k, bias, scoring, groups, top_groups, label="equal keys")


def test_many_tokens():
    x = logits_of(5000, 96, torch.bfloat16)
    got = fq.moe_route(x, 4)
    check(x, got, 4, label="many")
