"""moe_dispatch: places and rows equal a stable sort's; moe_combine against
float64.  One and several launches, odd widths, padding, repeated experts."""
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


def choices(tokens, top_k, experts, seed=0, padding=False, skew=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + tokens)
    u = torch.rand((tokens, top_k), generator=g, device="cuda") ** skew
    e = (u * experts).int().clamp(max=experts - 1)
    if padding:
        e[torch.rand((tokens, top_k), generator=g, device="cuda") < 0.2] = -1
        if tokens > 3:
            e[2] = experts        # past the last: no row
            e[3] = -2 ** 31
    return e


def check(x, e, experts, got):
    rows, off, place = got
    want_off, want_place = lu.dispatch(e.cpu().numpy(), experts)
    assert off.dtype is torch.int64 and place.dtype is torch.int32
    assert np.array_equal(off.cpu().numpy(), want_off)
    assert np.array_equal(place.cpu().numpy(), want_place)
    token, choice = np.nonzero(want_place >= 0)
    at = torch.from_numpy(want_place[token, choice]).cuda()
    assert torch.equal(rows[at].view(torch.int16), x[torch.from_numpy(token).cuda()].view(torch.int16))


# up to 8192 choices in one launch (workgroups of several tokens from 1025 on), more in several;
# passes of 1024
@pytest.mark.parametrize("tokens,top_k", [(1, 1), (1, 64), (3, 5), (64, 8), (511, 8), (512, 8), (513, 8), (4097, 1),
                                          (700, 6), (64, 64), (2500, 7), (20000, 2)])
@pytest.mark.parametrize("experts", [1, 2, 31, 64, 257, 1024])
@pytest.mark.parametrize("padding", [False, True])
def test_dispatch(tokens, top_k, experts, padding):
    e = choices(tokens, top_k, experts, padding=padding, skew=2.0)
    x = torch.randn((tokens, 24), device="cuda").bfloat16()
    check(x, e, experts, fq.moe_dispatch(x, e, experts))


@pytest.mark.parametrize("hidden", [1, 2, 7, 8, 16, 100, 1999, 2048, 7168])
@pytest.mark.parametrize("tokens", [5, 1200])
def test_widths(hidden, tokens):
    e = choices(tokens, 4, 16)
    x = torch.randn((tokens, hidden), device="cuda").bfloat16()
    check(x, e, 16, fq.moe_dispatch(x, e, 16))


def test_chunks_of_several_passes():
    # more than 256 chunks of 1024 choices
    for tokens, top_k, experts in ((150001, 2, 37), (400000, 1, 1024), (70000, 8, 8)):
        e = choices(tokens, top_k, experts, padding=True, skew=3.0)
        x = torch.arange(tokens, device="cuda").int().view(torch.bfloat16).view(tokens, 2)
        check(x, e, experts, fq.moe_dispatch(x, e, experts))


def test_all_to_one_expert_and_none():
    for tokens in (10, 3000):
        x = torch.randn((tokens, 16), device="cuda").bfloat16()
        e = torch.full((tokens, 3), 5, dtype=torch.int32, device="cuda")
        check(x, e, 9, fq.moe_dispatch(x, e, 9))
        e.fill_(-1)
        out = (torch.full((3 * tokens, 16), 2.0, device="cuda").bfloat16(),
               torch.full((10,), 7, dtype=torch.int64, device="cuda"),
               torch.full((tokens, 3), 7, dtype=torch.int32, device="cuda"))
        rows, off, place = fq.moe_dispatch(x, e, 9, out=out)
        assert rows.data_ptr() == out[0].data_ptr()
        assert (rows == 2).all() and (off == 0).all() and (place == -1).all()


def test_no_tokens():
    rows, off, place = fq.moe_dispatch(torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda"),
                                       torch.zeros((0, 4), dtype=torch.int32, device="cuda"), 300)
    assert rows.shape == (0, 64) and place.shape == (0, 4) and off.tolist() == [0] * 301


def test_rows_past_the_last_stay():
    for tokens in (50, 2000):
        x = torch.randn((tokens, 40), device="cuda").bfloat16()
        e = choices(tokens, 4, 11, padding=True)
        out = (torch.full((4 * tokens, 40), 2.0, device="cuda").bfloat16(),
               torch.empty(12, dtype=torch.int64, device="cuda"),
               torch.empty((tokens, 4), dtype=torch.int32, device="cuda"))
        rows, off, _ = fq.moe_dispatch(x, e, 11, out=out)
        check(x, e, 11, out)
        assert (rows[int(off[-1]):] == 2).all()


def test_odd_alignment():
    for tokens in (9, 1500):
        base = torch.randn(tokens * 64 + 1, device="cuda").bfloat16()
        x = base[1:].view(tokens, 64)
        e = choices(tokens, 4, 8)
        check(x, e, 8, fq.moe_dispatch(x, e, 8))
        y = torch.randn(4 * tokens * 64 + 1, device="cuda").bfloat16()[1:].view(4 * tokens, 64)
        place = fq.moe_dispatch(x, e, 8)[2]
        w = torch.rand((tokens, 4), device="cuda")
        assert torch.equal(fq.moe_combine(y, place, w), fq.moe_combine(y.clone(), place, w))


def combined(y, place, w, add):
    y, w, p = lu.f64(y), lu.f64(w), place.cpu().numpy()
    ok = (p >= 0) & (p < len(y))
    terms = np.where(ok[..., None], np.where(ok, w, 0)[..., None] * y[np.where(ok, p, 0)], 0.0)
    total = terms.sum(1) + (0 if add is None else lu.f64(add))
    mag = np.abs(terms).sum(1) + (0 if add is None else np.abs(lu.f64(add)))
    return total, mag


@pytest.mark.parametrize("n", [1, 5, 8, 64, 1999, 2048, 7168])
@pytest.mark.parametrize("y_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("out_dtype", [None, torch.float32])
@pytest.mark.parametrize("with_add", [False, True])
def test_combine(n, y_dtype, out_dtype, with_add):
    for tokens, top_k in ((1, 1), (33, 8), (70, 3)):
        e = choices(tokens, top_k, 9, padding=tokens == 33)
        place = torch.from_numpy(lu.dispatch(e.cpu().numpy(), 9)[1].astype(np.int32)).cuda()
        y = torch.randn((tokens * top_k, n), device="cuda").to(y_dtype)
        w = torch.rand((tokens, top_k), device="cuda")
        add = torch.randn((tokens, n), device="cuda").bfloat16() if with_add else None
        out = fq.moe_combine(y, place, w, add=add, out_dtype=out_dtype)
        assert out.dtype is (out_dtype or torch.bfloat16)
        want, mag = combined(y, place, w, add)
        # top_k products and sums in FP32
        bound = (2 * top_k + 1) * lu.FP32 * mag + 1e-37
        if out.dtype is torch.bfloat16:
            bound = bound + lu.BF16 * (np.abs(want) + bound)
        lu.check(lu.f64(out), want, bound, "%d tokens" % tokens)


def test_combine_in_place_and_outside_places():
    y = torch.randn((12, 64), device="cuda").bfloat16()
    y[7] = math.nan
    place = torch.tensor([[0, -1], [3, 12], [5, 2 ** 31 - 1], [-2 ** 31, 11], [-1, 40]], dtype=torch.int32,
                         device="cuda")
    w = torch.tensor([[0.5, math.nan], [1.0, math.inf], [2.0, math.nan], [math.inf, 0.25], [math.nan, 1.0]],
                     device="cuda")
    add = torch.randn((5, 64), device="cuda").bfloat16()
    want, mag = combined(y, place, w, add)
    got = fq.moe_combine(y, place, w, add=add)
    lu.check(lu.f64(got), want, (5 * lu.FP32 + lu.BF16) * mag * 1.01 + 1e-37, "outside")
    fq.moe_combine(y, place, w, add=add, out=add)
    assert torch.equal(add, got)
    # the same row twice, and a row that is not finite where it is asked for
    place = torch.tensor([[3, 3], [7, 0]], dtype=torch.int32, device="cuda")
    out = fq.moe_combine(y, place, torch.ones((2, 2), device="cuda"), out_dtype=torch.float32)
    assert torch.equal(out[0], 2 * y[3].float()) and torch.isnan(out[1]).all()
    none = fq.moe_combine(y[:0], place, torch.ones((2, 2), device="cuda"))
    assert (none == 0).all() and none.shape == (2, 64)


def test_there_and_back():
    # every row comes back with the sum of its weights
    for tokens in (31, 3000):
        x = torch.randn((tokens, 128), device="cuda").bfloat16()
        w, e = fq.moe_route(torch.randn((tokens, 24), device="cuda"), 4)
        rows, off, place = fq.moe_dispatch(x, e, 24)
        back = fq.moe_combine(rows, place, w, out_dtype=torch.float32)
        assert torch.allclose(back, x.float(), rtol=1e-5, atol=1e-6)


def test_rows_that_the_caches_do_not_hold():
    # 256 MiB and more there, 64 MiB and more back; a choice in five without a row
    tokens, top_k, experts, hidden = 4500, 2, 9, 16384
    e = choices(tokens, top_k, experts, padding=True)
    x = torch.randn((tokens, hidden), device="cuda").bfloat16()
    rows, off, place = fq.moe_dispatch(x, e, experts)
    check(x, e, experts, (rows, off, place))
    # weights that are powers of two: the sums are exact but for one rounding
    w = torch.tensor([0.5, 2.0], device="cuda").expand(tokens, 2).contiguous()
    want = sum(w[:, j:j + 1] * (place[:, j:j + 1] >= 0) * x.float() for j in range(2)).bfloat16()
    assert torch.equal(fq.moe_combine(rows, place, w), want)


def test_past_32_bit_offsets():
    # rows beyond 2^31 elements
    tokens, top_k, hidden = 70, 8, 1 << 22
    x = torch.empty((tokens, hidden), dtype=torch.bfloat16, device="cuda")
    x.copy_(torch.arange(tokens, device="cuda")[:, None].expand(tokens, hidden))
    x[:, -1] = -x[:, 0]
    e = choices(tokens, top_k, 5)
    rows, off, place = fq.moe_dispatch(x, e, 5)
    want_off, want = lu.dispatch(e.cpu().numpy(), 5)
    assert np.array_equal(place.cpu().numpy(), want)
    flat = place.view(-1).long()
    token = torch.arange(tokens, device="cuda").repeat_interleave(top_k)
    for c in (0, 1, hidden // 2, hidden - 2, hidden - 1):
        assert torch.equal(rows[flat, c], x[token, c])
    out = fq.moe_combine(rows, place, torch.full((tokens, top_k), 0.125, device="cuda"))
    for c in (0, 1, hidden // 2, hidden - 2, hidden - 1):
        assert torch.equal(out[:, c], x[:, c])
