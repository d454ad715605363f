"""nvfp4_kv_append and nvfp4_kv_read on the GPU: the cache's bytes equal the
oracle's nvfp4_quantize of the same rows bit for bit, places that no slot
names keep their contents, and reads equal the oracle's dequant."""
import numpy as np
import pytest
import torch

import fp4_block_quantization_amd as fq
import oracle
import workloads
from gpuutil import Guards, assert_same, bits_of, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.rollout_lib()


def make_cache(gu, pages, page, heads, dim):
    """A cache inside guard bytes, filled with 0x5A."""
    u8, f32 = torch.uint8, torch.float32
    c = fq.NvFp4KvCache(gu.empty((pages, heads, page, dim // 2), u8),
                        gu.empty((pages, heads, page, dim // 16), u8),
                        gu.empty((pages, heads, page), f32),
                        gu.empty((pages, heads, page, dim // 2), u8),
                        gu.empty((pages, heads, dim // 16, page), u8),
                        gu.empty((pages, heads, page), f32))
    for t in c:
        t.view(torch.uint8).fill_(0x5A)
    return c


def rows_of(cache):
    """The cache's host arrays with one row per [slot, head]: codes, scales, s."""
    out = []
    for i in (0, 3):
        codes, scales, ts = (t.cpu().numpy() for t in cache[i:i + 3])
        if i:
            scales = scales.transpose(0, 1, 3, 2)
        by_slot = [np.ascontiguousarray(a.swapaxes(1, 2)).reshape(-1, a.shape[1], *a.shape[3:])
                   for a in (codes, scales, ts)]
        out.append(by_slot)
    return out


def inputs(seed, tokens, heads, dim):
    x = workloads.random_rows(seed, tokens * heads, dim, dist=1, row_gain_sigma=1.0)
    if tokens > 2:  # a zero row, signed zeros, the largest and smallest values
        x[0] = 0
        x[1, ::2] = 0x8000
        x[2, :3] = (0x7F7F, 0x0001, 0x8080)
        x[3, :] = 0x0001
    return x


SHAPES = [(1, 16, 1, 16), (5, 16, 1, 64), (37, 16, 8, 128), (64, 64, 2, 256), (33, 48, 3, 80),
          (17, 32, 5, 112), (130, 16, 2, 512), (9, 128, 7, 192), (41, 16, 2, 48)]


@pytest.mark.parametrize("fos", [True, False])
@pytest.mark.parametrize("tokens,page,heads,dim", SHAPES)
def test_append_and_read_equal_the_oracle(tokens, page, heads, dim, fos):
    rng = np.random.default_rng(tokens * 1000 + dim)
    gu = Guards()
    pages = -(-tokens // page) + 2
    cache = make_cache(gu, pages, page, heads, dim)
    slots = rng.permutation(pages * page)[:tokens].astype(np.int64)
    kb, vb = (inputs(s, tokens, heads, dim) for s in (7 * tokens + dim, 7 * tokens + dim + 1))
    k, v = (to_dev(b).view(tokens, heads, dim) for b in (kb, vb))
    dev_slots = torch.from_numpy(slots).cuda()
    fq.nvfp4_kv_append(cache, k, v, dev_slots, four_over_six=fos)
    gu.check("append")
    order = rng.permutation(tokens)
    out = (gu.empty((tokens, heads, dim), torch.bfloat16),
           gu.empty((tokens, heads, dim), torch.bfloat16))
    got = fq.nvfp4_kv_read(cache, dev_slots[torch.from_numpy(order).cuda()].contiguous(), out=out)
    gu.check("read")
    others = np.setdiff1d(np.arange(pages * page), slots)
    for (codes, scales, ts), bits, back, name in zip(rows_of(cache), (kb, vb), got, "kv"):
        want = oracle.nvfp4_quantize(bits, four_over_six=fos)
        assert_same(codes[slots].reshape(-1, dim // 2), want[0], name + " codes")
        assert_same(scales[slots].reshape(-1, dim // 16), want[1], name + " scales")
        assert_same(ts[slots].reshape(1, -1), want[2][None], name + " token scales")
        for a in (codes, scales, ts):
            assert (np.ascontiguousarray(a[others]).view(np.uint8) == 0x5A).all(), name
        assert_same(bits_of(back).reshape(tokens, heads * dim),
                    want[3].reshape(tokens, heads * dim)[order], name + " read")


def test_every_finite_value_and_scaled_rows():
    # every finite BF16 pattern, ordered by magnitude, in rows of 128
    p = np.arange(0x7F80, dtype=np.uint16)
    bits = np.stack([p, p | 0x8000], 1).reshape(-1, 128)
    tokens = bits.shape[0]
    gu = Guards()
    pages = -(-tokens // 16)
    for fos in (True, False):
        cache = make_cache(gu, pages, 16, 1, 128)
        x = to_dev(bits).view(tokens, 1, 128)
        slots = torch.arange(tokens, device="cuda")
        fq.nvfp4_kv_append(cache, x, x, slots, four_over_six=fos)
        k, v = fq.nvfp4_kv_read(cache, slots)
        gu.check("every value")
        want = oracle.nvfp4_quantize(bits, four_over_six=fos)
        for codes, scales, ts in rows_of(cache):
            assert_same(codes.reshape(-1, 64)[:tokens], want[0], "codes")
            assert_same(scales.reshape(-1, 8)[:tokens], want[1], "scales")
            assert_same(ts.reshape(1, -1)[:, :tokens], want[2][None], "token scales")
        for t in (k, v):
            assert_same(bits_of(t).reshape(-1, 128), want[3], "read")


def test_strided_rows_skipped_slots_and_streams():
    tokens, heads, dim, page = 21, 2, 64, 16
    gu = Guards()
    cache = make_cache(gu, 3, page, heads, dim)
    fused = to_dev(workloads.random_rows(5, tokens, 7 * dim)).view(tokens, 7 * dim)
    k = fused[:, 3 * dim:5 * dim].view(tokens, heads, dim)
    v = fused[:, 5 * dim:].view(tokens, heads, dim)
    slots = torch.arange(tokens, device="cuda") * 2
    slots[3], slots[7], slots[9] = -1, 3 * page, 1 << 40
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fq.nvfp4_kv_append(cache, k, v, slots)
        rk, rv = fq.nvfp4_kv_read(cache, slots)
    side.synchronize()
    gu.check("strided")
    keep = np.ones(tokens, bool)
    keep[[3, 7, 9]] = False
    for src, back, (codes, _, ts) in zip((k, v), (rk, rv), rows_of(cache)):
        want = oracle.nvfp4_quantize(bits_of(src.contiguous()).reshape(-1, dim))[3]
        want = want.reshape(tokens, -1).copy()
        want[~keep] = 0
        assert_same(bits_of(back).reshape(tokens, -1), want, "read")
        used = slots.cpu().numpy()[keep]
        others = np.setdiff1d(np.arange(3 * page), used)
        assert (codes[others] == 0x5A).all()
        assert (np.ascontiguousarray(ts[others]).view(np.uint8) == 0x5A).all()


def test_empty_calls_and_refusals():
    cache = fq.nvfp4_kv_cache(2, 16, 2, 64)
    none = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    fq.nvfp4_kv_append(cache, none, none, slots)
    k, v = fq.nvfp4_kv_read(cache, slots)
    assert k.shape == v.shape == (0, 2, 64)
    one = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    four = torch.zeros(4, dtype=torch.int64, device="cuda")
    bad = [dict(k=one.float()), dict(slots=four.int()), dict(slots=four[:3]),
           dict(k=one.transpose(1, 2)), dict(v=one[:3]), dict(k=one.repeat(1, 1, 2)[..., ::2]),
           dict(cache=cache[:5]), dict(cache=(cache[0][:1], *cache[1:])),
           dict(k=one.cpu()), dict(four_over_six=2),
           dict(k=torch.zeros(4 * 128 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(4, 2, 64))]
    for kw in bad:
        args = dict(cache=cache, k=one, v=one, slots=four)
        args.update(kw)
        with pytest.raises(fq.Fp4qError):
            fq.nvfp4_kv_append(args["cache"], args["k"], args["v"], args["slots"],
                               four_over_six=args.get("four_over_six", True))
    with pytest.raises(fq.Fp4qError):
        fq.nvfp4_kv_read(cache, four, out=(one, one[:3]))
    for t in cache:
        assert not t.view(torch.uint8).any()  # a refused call writes nothing
