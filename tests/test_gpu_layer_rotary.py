"""rotary: queries and keys against float64, at head layouts, types, strides and
positions where it can go wrong; the inverse as the transposed map."""
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


def heads(tokens, n, d, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((tokens, n, d), generator=g, device="cuda").to(dtype)


def positions_of(tokens, start, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return start + torch.randint(0, max(1, 2 * tokens), (tokens,), generator=g, device="cuda")


def check(q, k, pos, f, amplitude, interleaved, inverse, got, label):
    for x, y, name in ((q, got[0], "q"), (k, got[1], "k")):
        if x is None:
            assert y is None
            continue
        assert y.dtype is x.dtype and y.shape == x.shape
        want, bound = lu.rotary(lu.f64(x), pos.cpu().numpy(), lu.f64(f), amplitude, interleaved, inverse,
                                x.dtype is torch.bfloat16)
        lu.check(lu.f64(y), want, bound, "%s %s" % (label, name))


# head_dim, dims: whole heads, parts of heads, halves that are not whole 16 bytes, one pair
LAYOUTS = [(128, 128), (64, 64), (256, 256), (192, 64), (80, 80), (96, 26), (72, 36), (7, 4), (2, 2)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("d,dims", LAYOUTS)
def test_layouts(d, dims, interleaved, inverse, dtype):
    for tokens, hq, hk in ((1, 1, 0), (5, 3, 1), (67, 8, 2)):
        q, k = heads(tokens, hq, d, dtype, 1), heads(tokens, hk, d, dtype, 2) if hk else None
        f, a = fq.rotary_frequencies(dims, method="parts", factor=8.0, original_positions=2048)
        pos = positions_of(tokens, 3000)
        got = fq.rotary(q, k, pos, f, amplitude=a, interleaved=interleaved, inverse=inverse)
        check(q, k, pos, f, a, interleaved, inverse, got, "%d tokens" % tokens)


@pytest.mark.parametrize("start", [0, 1 << 20, 2 ** 31 - 70, 2 ** 40, -5000])
def test_far_and_negative_positions(start):
    q = heads(33, 4, 64, torch.float32, 3)
    f, _ = fq.rotary_frequencies(64)
    pos = positions_of(33, start)
    got = fq.rotary(q, None, pos, f)
    check(q, None, pos, f, 1.0, False, False, got, "from %d" % start)


def test_exact_quarters():
    # a quarter, a half and three quarters of a turn to every side, and whole turns
    q = heads(9, 1, 2, torch.float32, 4)
    f = torch.tensor([np.pi / 2], dtype=torch.float64, device="cuda")
    pos = torch.arange(-4, 5, device="cuda")
    got = fq.rotary(q, None, pos, f)
    check(q, None, pos, f, 1.0, False, False, got, "quarters")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad", [0, 1])  # 1: rows that are not whole 16 bytes apart
@pytest.mark.parametrize("interleaved", [False, True])
def test_strided_in_place_and_out(dtype, pad, interleaved):
    tokens, hq, hk, d, dims = 19, 6, 2, 64, 32
    qkv = torch.randn((tokens, (hq + 2 * hk) * d + pad), device="cuda").to(dtype)
    rows = qkv[:, :(hq + 2 * hk) * d].unflatten(1, (-1, d))
    q, k, v = rows.split([hq, hk, hk], 1)
    f, _ = fq.rotary_frequencies(dims)
    pos = positions_of(tokens, 100)
    want = fq.rotary(q, k, pos, f, interleaved=interleaved)
    check(q, k, pos, f, 1.0, interleaved, False, want, "strided")
    # written into slices of another tensor: nothing else of it changes
    other = torch.full_like(qkv, 7.0)
    oq, ok, ov = other[:, :(hq + 2 * hk) * d].unflatten(1, (-1, d)).split([hq, hk, hk], 1)
    got = fq.rotary(q, k, pos, f, interleaved=interleaved, out=(oq, ok))
    assert got[0].data_ptr() == oq.data_ptr() and got[1].data_ptr() == ok.data_ptr()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert (ov == 7).all() and (other[:, (hq + 2 * hk) * d:] == 7).all()
    # in place: the values, and what the heads do not turn, stay as they are
    before = qkv.clone()
    fq.rotary(q, k, pos, f, interleaved=interleaved, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    was = before[:, :(hq + 2 * hk) * d].unflatten(1, (-1, d))
    assert torch.equal(rows[..., dims:], was[..., dims:]) and torch.equal(v, was[:, hq + hk:])
    assert torch.equal(qkv[:, (hq + 2 * hk) * d:], before[:, (hq + 2 * hk) * d:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_many_tokens_are_as_few(dtype, interleaved, inverse):
    # over 64 MiB at once, and in pieces below that
    tokens = 9001
    x = heads(tokens, 20, 192, dtype, 51)
    f, a = fq.rotary_frequencies(64, method="parts", factor=8.0, original_positions=2048)
    pos = positions_of(tokens, 100)
    kw = dict(amplitude=a, interleaved=interleaved, inverse=inverse)
    few = [fq.rotary(x[i:i + 1500, :16], x[i:i + 1500, 16:], pos[i:i + 1500], f, **kw) for i in range(0, tokens, 1500)]
    want = torch.cat([q for q, _ in few]), torch.cat([k for _, k in few])
    check(x[:50, :16], x[:50, 16:], pos[:50], f, a, interleaved, inverse, (want[0][:50], want[1][:50]), "few")
    got = fq.rotary(x[:, :16], x[:, 16:], pos, f, **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    fq.rotary(x[:, :16], x[:, 16:], pos, f, out=(x[:, :16], x[:, 16:]), **kw)
    assert torch.equal(x[:, :16], want[0]) and torch.equal(x[:, 16:], want[1])


def test_inverse_is_the_transposed_map():
    # <rotary(x), y> = <x, rotary^T(y)>, with an amplitude; and against differences of the forward
    d, tokens = 32, 7
    f, _ = fq.rotary_frequencies(24)
    pos = positions_of(tokens, 50)
    x, y = (heads(tokens, 3, d, torch.float32, s) for s in (5, 6))
    fx = fq.rotary(x, None, pos, f, amplitude=1.25)[0]
    ty = fq.rotary(y, None, pos, f, amplitude=1.25, inverse=True)[0]
    a, b = (fx.double() * y.double()).sum().item(), (x.double() * ty.double()).sum().item()
    mag = (fx.double() * y.double()).abs().sum().item() + (x.double() * ty.double()).abs().sum().item()
    assert abs(a - b) <= mag * 1.5 * 8 * 2.0 ** -23
    for i in (0, 5, 13, 30):  # a linear map: a step of one element gives the gradient's column exactly
        step = torch.zeros_like(x)
        step[2, 1, i] = 1.0
        col = fq.rotary(step, None, pos, f, amplitude=1.25)[0]
        assert abs((col.double() * y.double()).sum().item() - ty[2, 1, i].item()) <= 1e-5


def test_leading_dimensions_empty_and_repeats():
    f, _ = fq.rotary_frequencies(64)
    q = torch.randn((3, 5, 4, 64), device="cuda").bfloat16()
    k = torch.randn((3, 5, 2, 64), device="cuda").bfloat16()
    pos = positions_of(15, 9).view(3, 5)
    got = fq.rotary(q, k, pos, f)
    assert got[0].shape == q.shape and got[1].shape == k.shape
    flat = fq.rotary(q.view(15, 4, 64), k.view(15, 2, 64), pos.view(-1), f)
    for a, b in zip(got, flat):
        assert torch.equal(a.view_as(b), b)
    none = fq.rotary(q[:0], k[:0], pos[:0], f)
    assert none[0].shape == (0, 5, 4, 64)


def test_infinities_and_nans_stay_in_their_pairs():
    f, _ = fq.rotary_frequencies(16)
    x = heads(2, 2, 16, torch.float32, 8)
    clean = fq.rotary(x, None, torch.tensor([3, 4], device="cuda"), f)[0]
    x[0, 1, 3], x[1, 0, 9] = float("nan"), float("inf")
    got = fq.rotary(x, None, torch.tensor([3, 4], device="cuda"), f)[0]
    bad = torch.zeros_like(x, dtype=torch.bool)
    bad[0, 1, 3] = bad[0, 1, 11] = bad[1, 0, 9] = bad[1, 0, 1] = True
    assert torch.equal(got[~bad], clean[~bad])
    assert not torch.isfinite(got[bad]).any()


def test_past_32_bit_offsets():
    # the last token's row begins beyond 2^31 elements
    tokens, stride = 5, 1 << 29
    big = torch.empty((tokens - 1) * stride + 256, dtype=torch.bfloat16, device="cuda")
    q = big.as_strided((tokens, 2, 128), (stride, 128, 1))
    src = heads(tokens, 2, 128, torch.bfloat16, 9)
    q.copy_(src)
    f, _ = fq.rotary_frequencies(128)
    pos = positions_of(tokens, 77)
    want = fq.rotary(src, None, pos, f)[0]
    assert torch.equal(fq.rotary(q, None, pos, f)[0], want)
    fq.rotary(q, None, pos, f, out=(q, None))
    assert torch.equal(q, want)
