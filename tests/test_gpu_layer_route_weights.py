"""moe_route's sigmoid weights where scores leave FP32's range: against the
logarithms of the scores in float64, which do not."""
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


def check(logits, weights, experts, renormalize, scale=1.0):
    """The weights of the chosen experts.  With t the largest min(x, 0) of a token's choices, each
    is exp(min(x, 0) - t) / (1 + exp(-|x|)) over their sum: the argument rounds (2^-24 of it), the
    two exponentials are off by 2 units each, and up to 4 + top_k additions and quotients round;
    what ends below FP32's normal numbers is off by a few of its smallest steps."""
    x = np.take_along_axis(lu.f64(logits), experts.cpu().numpy().astype(np.int64), 1)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        log_score = np.minimum(x, 0.0) - np.log1p(np.exp(-np.abs(x)))
        top = log_score.max(1, keepdims=True) if renormalize else np.zeros((len(x), 1))
        none = top == -math.inf
        w = np.exp(log_score - np.where(none, 0.0, top))
        if renormalize:
            w = w / np.where(none, 1.0, w.sum(1, keepdims=True))
        away = np.where(np.isfinite(x), np.abs(x - (np.where(none, 0.0, top) if renormalize else 0.0)), 0.0)
    rel = (np.minimum(away, 200.0) + 16 + x.shape[1]) * 2.0 ** -23
    lu.check(weights.cpu().numpy(), w * scale, w * scale * rel + 8 * scale * 2.0 ** -149, "weights")
    return w


ROWS = [[-88.0, -89.0, -90.0, -120.0], [-100.0, -101.0, -103.5, -104.0], [-200.0, -150.0, -300.0, -1000.0],
        [-1000.0, -1001.0, -1000.0, -5000.0], [-1e30, -1e30, -2e30, -3e38], [-3.3e38] * 4,
        [50.0, -95.0, -100.0, -110.0], [-math.inf, -300.0, -301.0, -math.inf], [-math.inf] * 4,
        [math.inf, 3.0, -90.0, -95.0], [0.0, -0.0, -88.5, 88.5], [-95.0, -95.0, -95.0, -95.0]]


@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows(dtype, with_bias):
    x = torch.tensor(ROWS, device="cuda").to(dtype)
    bias = torch.tensor([0.0, 0.1, 0.2, 0.3], device="cuda") if with_bias else None
    for top_k in (1, 2, 4):
        for renormalize in (True, False):
            w, e = fq.moe_route(x, top_k, bias=bias, scoring="sigmoid", renormalize=renormalize)
            want = check(x, w, e, renormalize)
            if renormalize:  # every token but the one without any score keeps its experts' sum
                assert np.allclose(w.sum(1).cpu().numpy(), want.sum(1), atol=1e-6)
                assert [i for i, s in enumerate(want.sum(1)) if s == 0] in ([8], [7, 8])


def test_the_weights_of_two_low_logits():
    x = torch.tensor([[-88.0, -89.0], [-100.0, -101.0], [-150.0, -200.0]], device="cuda")
    w, e = fq.moe_route(x, 2, scoring="sigmoid")
    assert e.tolist() == [[0, 1]] * 3
    p = 1.0 / (1.0 + math.exp(-1.0))
    want = torch.tensor([[p, 1.0 - p], [p, 1.0 - p], [1.0, math.exp(-50.0)]], dtype=torch.float64)
    assert torch.allclose(w.cpu().double(), want, rtol=1e-5, atol=0.0)


@pytest.mark.parametrize("experts,groups,top_groups,top_k", [(64, 1, 1, 8), (100, 1, 1, 64), (256, 8, 4, 8),
                                                              (1024, 1, 1, 10)])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("low", [-80.0, -95.0, -140.0, -700.0])
def test_low_logits(experts, groups, top_groups, top_k, with_bias, low):
    g = torch.Generator(device="cuda").manual_seed(experts)
    x = low + 6.0 * torch.randn((23, experts), generator=g, device="cuda")
    bias = torch.rand(experts, generator=g, device="cuda") if with_bias else None
    for renormalize in (True, False):
        w, e = fq.moe_route(x, top_k, bias=bias, scoring="sigmoid", groups=groups, top_groups=top_groups,
                            renormalize=renormalize, scale=2.5)
        check(x, w, e, renormalize, 2.5)
        if bias is None and groups == 1:
            order = x.sort(dim=1, descending=True, stable=True).indices[:, :top_k]
            assert torch.equal(e.long(), order)


def test_weights_beside_those_that_underflow():
    # what the softmax does with scores that leave the range, and the sigmoid's at the other end
    x = torch.tensor([[-200.0, -150.0, -300.0, -1000.0], [300.0, -300.0, 200.0, 0.0]], device="cuda")
    w, e = fq.moe_route(x, 2, scoring="sigmoid")
    assert e.tolist() == [[1, 0], [0, 2]] and w[1].tolist() == [0.5, 0.5]
    check(x, w, e, True)
    w, e = fq.moe_route(x, 2, renormalize=False)
    assert e.tolist() == [[1, 0], [0, 2]] and w[1, 0] == 1.0
    assert abs(w[1, 1].item() - math.exp(-100)) <= 2.0 ** -149
    bias = torch.tensor([0.0, 0.0, 5.0, 6.0], device="cuda")
    w, e = fq.moe_route(torch.tensor([[0.0, 0.0, -200.0, -200.0]], device="cuda"), 2, bias=bias)
    assert e.tolist() == [[3, 2]] and w.tolist() == [[0.5, 0.5]]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_the_weight_of_the_one_expert_that_is_not_shut_off(scoring):
    x = torch.full((1, 40), -math.inf, device="cuda")
    x[0, 0] = 0.75
    for renormalize in (True, False):
        w, e = fq.moe_route(x, 6, scoring=scoring, renormalize=renormalize)
        assert e.tolist() == [[0, 1, 2, 3, 4, 5]]
        one = 1.0 if renormalize or scoring == "softmax" else 1.0 / (1.0 + math.exp(-0.75))
        assert abs(w[0, 0].item() - one) <= 2.0 ** -22 and (w[0, 1:] == 0).all()
