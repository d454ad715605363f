"""The rollout binding's checks: tensors that hold the right number of
elements in another shape are refused, not misread, and so are inputs that
ask for a gradient."""
import pytest
import torch

import fp4_block_quantization_amd as fq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.rollout_lib()


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8, device="cuda")


def f32(*s):
    return torch.zeros(s, device="cuda")


def bf16(*s):
    return torch.zeros(s, dtype=torch.bfloat16, device="cuda")


def ints(dtype, *s):
    return torch.zeros(s, dtype=dtype, device="cuda")


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("mx", [False, True])
def test_linear_shapes(mx, grouped):
    lead = (3,) if grouped else ()
    block = 32 if mx else 16
    good = dict(x=bf16(6, 64), codes=u8(*lead, 8, 32), scales=u8(*lead, 8, 64 // block))
    if not mx:
        good.update(block_scales=good.pop("scales"), row_scales=f32(*lead, 8))
    if grouped:
        good.update(offsets=ints(torch.int64, 4))
    call = fq.mxfp4_linear if mx else fq.nvfp4_linear
    call(**good)
    call(**good, out=bf16(6, 8))
    scales = "scales" if mx else "block_scales"
    bad = [{scales: good[scales].transpose(-1, -2).contiguous()}, {scales: good[scales].view(-1)},
           dict(out=bf16(8, 6)), dict(out=bf16(48)), dict(out=f32(2, 3, 8))]
    if not mx:
        bad += [dict(row_scales=f32(*lead, 2, 4)), dict(row_scales=f32(*lead, 8, 1))]
    if grouped:
        bad += [dict(offsets=ints(torch.int64, 2, 2)), {scales: good[scales].view(24, -1)}]
    for kw in bad:
        with pytest.raises(fq.Fp4qError):
            call(**{**good, **kw})


def test_cache_shapes():
    # 4 pages of 32 tokens of 2 heads of 64
    cache = fq.nvfp4_kv_cache(4, 32, 2, 64)
    slots, table = ints(torch.int64, 3), ints(torch.int32, 3, 2)
    row = bf16(3, 2, 64)
    swapped = {
        "value scales laid out like key scales": (4, u8(4, 2, 32, 4)),
        "key scales laid out like value scales": (1, u8(4, 2, 4, 32)),
        "heads and pages": (0, u8(2, 4, 32, 32)),
        "pages and heads of the values": (3, u8(2, 4, 32, 32)),
        "token scales by page": (2, f32(4, 64)),
        "token scales flat": (5, f32(256)),
    }
    for what, (i, t) in swapped.items():
        bad = list(cache)
        bad[i] = t
        assert bad[i].numel() == cache[i].numel()
        for call in (lambda c: fq.nvfp4_kv_append(c, row, row, slots),
                     lambda c: fq.nvfp4_kv_read(c, slots),
                     lambda c: fq.nvfp4_kv_attention(row, c, table, ints(torch.int32, 3))):
            try:
                call(bad)
            except fq.Fp4qError:
                continue
            raise AssertionError("not refused: " + what)
    with pytest.raises(fq.Fp4qError):
        fq.nvfp4_kv_read(cache, slots, out=(bf16(3, 2, 64), bf16(2, 3, 64)))
    with pytest.raises(fq.Fp4qError):
        fq.nvfp4_kv_read(cache, slots, out=(bf16(3, 128), bf16(3, 128)))


def test_attention_shapes():
    cache = fq.nvfp4_kv_cache(4, 32, 2, 64)
    q, table, lens = bf16(2, 3, 4, 64), ints(torch.int32, 2, 2), ints(torch.int32, 2)
    prefix = (ints(torch.int32, 3, 1), ints(torch.int32, 3), ints(torch.int32, 4))
    fq.nvfp4_kv_attention(q, cache, table, lens, prefix=prefix, out=torch.empty_like(q))
    for kw in (dict(out=bf16(2, 4, 3, 64)), dict(out=bf16(2, 3, 256)), dict(seq_lens=lens[None]),
               dict(prefix=(prefix[0], prefix[1][None], prefix[2])),
               dict(prefix=(prefix[0], prefix[1], prefix[2].view(2, 2)))):
        with pytest.raises(fq.Fp4qError):
            fq.nvfp4_kv_attention(**{**dict(q=q, cache=cache, page_table=table, seq_lens=lens), **kw})


def test_gradients_are_refused():
    cache = fq.nvfp4_kv_cache(4, 32, 2, 64)
    slots, table, lens = ints(torch.int64, 3), ints(torch.int32, 3, 2), ints(torch.int32, 3)
    w = (u8(8, 32), u8(8, 4), f32(8))
    mxw = (u8(8, 32), u8(8, 2))
    asks = lambda t: t.clone().requires_grad_()
    x, row, q = bf16(6, 64), bf16(3, 2, 64), bf16(3, 4, 64)
    learnt = cache._replace(k_token_scales=asks(cache.k_token_scales))
    calls = [lambda: fq.nvfp4_linear(asks(x), *w), lambda: fq.mxfp4_linear(asks(x), *mxw),
             lambda: fq.nvfp4_linear(x, w[0], w[1], asks(w[2])),
             lambda: fq.nvfp4_linear(asks(x) * 2, *w),  # not a leaf
             lambda: fq.nvfp4_kv_append(cache, asks(row), row, slots),
             lambda: fq.nvfp4_kv_append(cache, row, asks(row), slots),
             lambda: fq.nvfp4_kv_attention(asks(q), cache, table, lens),
             lambda: fq.nvfp4_kv_attention(q, learnt, table, lens),
             lambda: fq.nvfp4_kv_read(learnt, slots)]
    for call in calls:
        with pytest.raises(fq.Fp4qError, match="gradient"):
            call()
        with torch.no_grad():
            call()
        with torch.inference_mode():
            call()
    assert not fq.nvfp4_linear(asks(x).detach(), *w).requires_grad


@pytest.mark.parametrize("mx", [False, True])
def test_out_and_out_dtype(mx):
    x, w = bf16(6, 64), (u8(8, 32), u8(8, 2)) if mx else (u8(8, 32), u8(8, 4), f32(8))
    call = fq.mxfp4_linear if mx else fq.nvfp4_linear
    assert call(x, *w).dtype is torch.bfloat16
    for dtype in (torch.bfloat16, torch.float32):
        out = torch.empty((6, 8), dtype=dtype, device="cuda")
        assert call(x, *w, out_dtype=dtype).dtype is dtype
        assert call(x, *w, out=out).data_ptr() == out.data_ptr()
        assert call(x, *w, out_dtype=dtype, out=out).dtype is dtype
        other = torch.float32 if dtype is torch.bfloat16 else torch.bfloat16
        for wrong in (other, torch.float16):
            with pytest.raises(fq.Fp4qError):
                call(x, *w, out_dtype=wrong, out=out)
    with pytest.raises(fq.Fp4qError):
        call(x, *w, out_dtype=torch.float16)
    for kw in (dict(), dict(out_dtype=torch.float32)):
        with pytest.raises(fq.Fp4qError):
            call(x, *w, out=[1.0], **kw)


def test_a_cache_made_as_it_is_read():
    # its tensors live as long as the call: the outputs must not take their memory
    cache = fq.nvfp4_kv_cache(8, 32, 2, 64)
    rows = [torch.randn((256, 2, 64), device="cuda").bfloat16() for _ in range(2)]
    slots = torch.arange(256, device="cuda")
    fq.nvfp4_kv_append(cache, *rows, slots)
    want = fq.nvfp4_kv_read(cache, slots)
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([250], dtype=torch.int32, device="cuda")
    q = torch.randn((1, 4, 64), device="cuda").bfloat16()
    attended = fq.nvfp4_kv_attention(q, cache, table, lens)
    for _ in range(5):
        for a, b in zip(fq.nvfp4_kv_read((t.clone() for t in cache), slots), want):
            assert torch.equal(a, b)
        assert torch.equal(fq.nvfp4_kv_attention(q, (t.clone() for t in cache), table, lens), attended)
