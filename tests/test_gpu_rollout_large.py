"""The rollout operators at sizes whose element, byte and row offsets pass 32
bits.  A row of a product depends on its own activations and a column on its
own weights alone, and a cached row on its token: so a large tensor is made
of repetitions of a small one whose results are known (the small ones are
checked against float64 by the other tests, and here again on a few rows),
and every repetition must equal it bit for bit."""
import numpy as np
import pytest
import torch

import fp4_block_quantization_amd as fq
import rolloututil as ru
import workloads
from gpuutil import to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.rollout_lib()
    yield
    torch.cuda.empty_cache()


def weights(mx, n, k):
    bits = to_dev(workloads.random_rows(n + k, n, k, scale=0.02, row_gain_sigma=0.5))
    if mx:
        q = fq.mxfp4_resq_quantize(bits)[:2]
        return q, ru.mx_values(*(t.cpu().numpy() for t in q))
    q = fq.nvfp4_quantize(bits, dequant=False)[:3]
    return q, ru.nv_values(*(t.cpu().numpy() for t in q))


def repeated(t, times):
    """t over and over along its first dimension (no copy kernel over 2^31 elements)."""
    out = torch.empty((times,) + tuple(t.shape), dtype=t.dtype, device=t.device)
    for i in range(times):
        out[i] = t
    return out.view((times * t.shape[0],) + tuple(t.shape[1:]))


def check_repeats(y, axis_len, label):
    """y [times, axis_len, ..]: every repetition equals the first."""
    y = y.view((-1, axis_len) + tuple(y.shape[1:]))
    for i in range(1, y.shape[0]):
        assert torch.equal(y[i], y[0]), "%s: repetition %d" % (label, i)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("rows", [1, 2, 40])
def test_weights_past_four_gib(rows, mx):
    n, k, times = 128, 16384, 4200  # 4.4e9 bytes of codes
    q, w = weights(mx, n, k)
    x_bits = workloads.random_rows(rows, rows, k, dist=1)
    big = [repeated(t, times) for t in q]
    assert big[0].numel() > 2 ** 32
    linear = fq.mxfp4_linear if mx else fq.nvfp4_linear
    y = linear(to_dev(x_bits), *big, out_dtype=torch.float32)
    check_repeats(y.t().contiguous(), n, "columns")
    want, bound = ru.linear_bound(ru.bf16_values(x_bits), w, False)
    ru.check(y[:, -n:].cpu().numpy(), want, bound, "last columns")


@pytest.mark.parametrize("mx", [False, True])
def test_experts_past_four_gib(mx):
    n, k, experts = 128, 16384, 4200
    q, w = weights(mx, n, k)
    big = [repeated(t, experts).view((experts,) + tuple(t.shape)) for t in q]
    x_bits = workloads.random_rows(7, 3, k, dist=1)
    counts = np.zeros(experts, np.int64)
    counts[[0, 1, 2050, 4097, experts - 1]] = 3
    offsets = torch.from_numpy(np.concatenate([[0], counts.cumsum()])).cuda()
    linear = fq.mxfp4_linear if mx else fq.nvfp4_linear
    y = linear(to_dev(np.tile(x_bits, (5, 1))), *big, offsets=offsets, out_dtype=torch.float32)
    check_repeats(y, 3, "experts")
    want, bound = ru.linear_bound(ru.bf16_values(x_bits), w, False)
    ru.check(y[-3:].cpu().numpy(), want, bound, "last expert")


def test_activations_and_outputs_past_four_gib():
    # rows x k of 4.4e9 bytes, then rows x n
    for rows_each, times, n, k in ((512, 4200, 48, 1024), (512, 600, 8192, 64)):
        q, w = weights(False, n, k)
        x_bits = workloads.random_rows(k, rows_each, k, dist=1)
        x = repeated(to_dev(x_bits), times)
        assert max(x.numel(), rows_each * times * n) > 2 ** 31
        y = fq.nvfp4_linear(x, *q)
        del x
        check_repeats(y, rows_each, "rows of %d" % k)
        want, bound = ru.linear_bound(ru.bf16_values(x_bits[-8:]), w, True)
        ru.check(y[-8:].float().cpu().numpy(), want, bound, "last rows of %d" % k)


def test_cache_past_four_gib():
    # codes of 38 GB a side, scales of 4.8 GB: pages on both sides of every power of two
    heads, dim, page, pages = 8, 256, 64, 590000
    batch, lens = 4, [300, 64, 130, 1]
    rng = np.random.default_rng(5)

    def cache_of(n):
        def make(dtype, *shape):
            return torch.empty((n, heads) + shape, dtype=dtype, device="cuda")
        side = [(torch.uint8, (page, dim // 2)), (torch.uint8, (page, dim // 16)),
                (torch.float32, (page,))]
        values = [side[0], (torch.uint8, (dim // 16, page)), side[2]]
        return fq.NvFp4KvCache(*(make(d, *s) for d, s in side + values))

    per = 5
    small, large = cache_of(batch * per), cache_of(pages)
    assert large.k_scales.numel() > 2 ** 32
    # page ids around the ends and the offsets 2^31 and 2^32 of codes and of scales
    ids = [0, pages - 1, pages - 2]
    for bytes_a_page in (heads * page * dim // 2, heads * page * dim // 16):
        for limit in (2 ** 31, 2 ** 32):
            ids += [limit // bytes_a_page + i for i in (-1, 0, 1)]
    ids += list(rng.choice(np.setdiff1d(np.arange(pages), ids), batch * per - len(ids), False))
    table = rng.permutation(np.array(ids, np.int32)).reshape(batch, per)
    near = np.arange(batch * per, dtype=np.int32).reshape(batch, per)

    def slots_of(t):
        return torch.from_numpy(np.concatenate(
            [t[b][np.arange(n) // page].astype(np.int64) * page + np.arange(n) % page
             for b, n in enumerate(lens)])).cuda()

    tokens = sum(lens)
    k, v, q = (to_dev(workloads.random_rows(s, n, dim, row_gain_sigma=0.7)).view(-1, h, dim)
               for s, n, h in ((1, tokens * heads, heads), (2, tokens * heads, heads),
                               (3, batch * 16, 16)))
    results = []
    for cache, t in ((small, near), (large, table)):
        fq.nvfp4_kv_append(cache, k, v, slots_of(t))
        back = fq.nvfp4_kv_read(cache, slots_of(t))
        tab, n = torch.from_numpy(t).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
        one = fq.nvfp4_kv_attention(q, cache, tab, n, lse=True)
        # the first sequence's tokens as the prefix of all, cut into parts
        members = torch.tensor([0, batch], dtype=torch.int32, device="cuda")
        pre = fq.nvfp4_kv_attention(q, cache, tab, n, lse=True,
                                    prefix=(tab[:1].contiguous(), n[:1].contiguous(), members))
        results.append([*back, *one, *pre])
    for a, b in zip(*results):
        kind = torch.int16 if a.dtype == torch.bfloat16 else torch.int32
        assert torch.equal(a.view(kind), b.view(kind))
    # and the reads are the quantizer's values
    for got, src in zip(results[1], (k, v)):
        want = fq.nvfp4_quantize(src.reshape(-1, dim), dequant=True)[3]
        assert torch.equal(got.reshape(-1, dim).view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("rows,grouped", [(1, False), (5, False), (20, False), (40, True)])
def test_longest_rows(rows, grouped, mx):
    # k at its limit: only the last elements of x are not zero
    k, n, used = 2 ** 26, 40, 4096 + 96
    gen = torch.Generator(device="cuda").manual_seed(rows)
    codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda", generator=gen)
    scales = torch.full((n, k // (32 if mx else 16)), 120 if mx else 0x35, dtype=torch.uint8,
                        device="cuda")
    x_bits = workloads.random_rows(rows, rows, used, dist=1)
    x = torch.zeros((rows, k), dtype=torch.bfloat16, device="cuda")
    x[:, -used:] = to_dev(x_bits)
    q = [codes, scales] if mx else [codes, scales, torch.ones(n, device="cuda")]
    tail = [codes[:, -used // 2:].cpu().numpy(), scales[:, -used // (32 if mx else 16):].cpu().numpy()]
    w = ru.mx_values(*tail) if mx else ru.nv_values(*tail, np.ones(n))
    offsets = None
    if grouped:
        q = [t[None] for t in q]
        offsets = torch.tensor([0, rows], device="cuda")
    linear = fq.mxfp4_linear if mx else fq.nvfp4_linear
    y = linear(x, *q, offsets=offsets, out_dtype=torch.float32)
    want, bound = ru.linear_bound(ru.bf16_values(x_bits), w, False)
    ru.check(y.cpu().numpy(), want, bound, "k=2^26")
