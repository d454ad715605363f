"""nvfp4_kv_attention over values whose token scales lie far apart, and over
tokens that a query does not see: against attention in float64, with a bound
that knows nothing of the tokens that are not seen and of those without
weight."""
import numpy as np
import pytest
import torch

import fp4_block_quantization_amd as fq
import rolloututil as ru
import workloads
from gpuutil import to_dev
from test_gpu_rollout_attention import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.rollout_lib()


def rewrite(b, seq, k_gain, v_gain):
    """New rows for sequence seq; gains [tokens] for its keys and values, infinity among them
    for a row with an infinite element."""
    n = b.lens[seq]
    pair = []
    for i, gain in enumerate((k_gain, v_gain)):
        x = ru.bf16_values(workloads.random_rows(900 + 2 * seq + i, n * b.kv_heads, b.dim))
        g = np.repeat(np.broadcast_to(np.asarray(gain, np.float64), (n,)), b.kv_heads)
        x = x * np.where(np.isinf(g), 1.0, g)[:, None]
        x[np.isinf(g), 3] = np.inf
        bits = workloads.to_bf16_bits(x.astype(np.float32))
        pair.append(to_dev(bits).view(n, b.kv_heads, b.dim))
    fq.nvfp4_kv_append(b.cache, *pair, torch.from_numpy(b._slots(b.table[seq], n)).cuda())


def check(b, scale, label):
    """Every query that sees finite values only, against float64.  Its bound:
    rolloututil.attention's for FP32 scores and FP16 weights; and weights more than 2^23 below
    the largest product of probability and token scale that this query sees, on values of at
    most 2688 token scales, counted as lost."""
    got = b.run(scale=scale).float().cpu().numpy()
    b.host = [t.cpu().numpy() for t in b.cache]
    token_scales = b.host[5].swapaxes(1, 2).reshape(-1, b.kv_heads)
    rep = b.heads // b.kv_heads
    for i, n in enumerate(b.lens):
        rows = [(b.table[i], n)]
        for g, pn in enumerate(b.prefix_lens):
            if b.members[g] <= i < b.members[g + 1]:
                rows.insert(0, (b.ptable[g], pn))
        k, v = (np.concatenate(t) for t in zip(*(b._values(r, c) for r, c in rows)))
        vs = np.concatenate([token_scales[b._slots(r, c)] for r, c in rows])
        k, v, vs = (np.repeat(t, rep, 1) for t in (k, v, vs))
        for t in range(b.tokens):
            m = len(k) - n + max(0, n - b.tokens + 1 + t)
            where = "%s: sequence %d query %d of %d keys" % (label, i, t, m)
            if m == 0:
                assert not got[i, t].any(), where
                continue
            if not np.isfinite(vs[:m]).all():
                assert not np.isfinite(got[i, t]).any(), where
                continue
            q = ru.bf16_values(b.q_bits[i, t])
            s = np.einsum("hd,thd->ht", q, k[:m]) * scale
            mag = np.einsum("hd,thd->ht", np.abs(q), np.abs(k[:m])) * abs(scale)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            o = np.einsum("ht,thd->hd", p, v[:m])
            delta = (b.dim + 32) * 2.0 ** -23 * (mag.max(1) + 1.0)
            spread = np.einsum("ht,thd->hd", p, np.abs(v[:m]))
            bound = spread * (2.0 ** -10 + 4 * delta + (m + 8) * 2.0 ** -23)[:, None]
            largest = (p * vs[:m].T.astype(np.float64)).max(1)
            bound += (m * 2.0 ** -23 * 2688 * largest)[:, None] + 2.0 ** -8 * np.abs(o) + 2.0 ** -133
            ru.check(got[i, t], o, bound, where)


@pytest.mark.parametrize("dim,heads,kv_heads,max_pages", [
    (64, 4, 2, None), (128, 4, 2, None), (128, 34, 2, None), (256, 2, 1, None), (192, 2, 2, 150),
    (128, 8, 1, 150)])
@pytest.mark.parametrize("power", [20, 45, 100])
def test_values_far_apart_without_weight(power, dim, heads, kv_heads, max_pages):
    # tokens with huge values have keys that the queries shun, before and after the others
    b = Batch(60 + power, [200, 70, 331, 1], heads=heads, kv_heads=kv_heads, dim=dim,
              max_pages=max_pages)
    rng = np.random.default_rng(power)
    # one direction of the keys decides: queries have 8 there, shunned keys -64
    for i, n in enumerate(b.lens):
        big = rng.random(n) < (0.0, 0.3, 0.02, 0.0)[i]
        if i == 0:
            big[40:45] = True
            big[150:] = True
        rewrite(b, i, 0.25, np.where(big, 2.0 ** (power - 50), 2.0 ** -50))
        slots = b._slots(b.table[i], n)
        k, _ = fq.nvfp4_kv_read(b.cache, torch.from_numpy(slots).cuda())
        k[:, :, 5] = torch.from_numpy(np.where(big, -64.0, 1.0)).to(k)[:, None]
        v = fq.nvfp4_kv_read(b.cache, torch.from_numpy(slots).cuda())[1]
        fq.nvfp4_kv_append(b.cache, k, v, torch.from_numpy(slots).cuda())
    b.q_bits[..., 5] = workloads.to_bf16_bits(np.full((1, 1), 8.0, np.float32))[0, 0]
    check(b, 1.0, "shunned 2^%d" % power)


@pytest.mark.parametrize("gain", [2.0 ** 30, 2.0 ** 60, np.inf])
@pytest.mark.parametrize("dim,tokens,heads,max_pages", [
    (64, 3, 4, None), (128, 9, 4, None), (128, 40, 8, 150), (256, 5, 2, None), (64, 70, 2, None)])
def test_values_that_a_query_does_not_see(dim, tokens, heads, max_pages, gain):
    # the last token's values are huge, or infinite: the queries before it do not see them
    b = Batch(70 + tokens, [tokens, 130, 64 + tokens // 2, 200], tokens=tokens, heads=heads,
              kv_heads=2, dim=dim, max_pages=max_pages)
    for i, n in enumerate(b.lens):
        g = np.full(n, 2.0 ** -20)
        g[-1] *= gain
        rewrite(b, i, 1.0, g)
    with np.errstate(invalid="ignore"):
        check(b, 0.125, "unseen %g" % gain)


@pytest.mark.parametrize("gain", [2.0 ** -112, 2.0 ** -100, 2.0 ** 100, 2.0 ** 120])
def test_tiny_and_huge_values(gain):
    # token scales down to FP32's subnormals and up to 2^111
    b = Batch(80, [100, 1, 64], heads=4, kv_heads=2, dim=128)
    for i in range(3):
        rewrite(b, i, 1.0, gain)
    check(b, 0.1, "gain %g" % gain)


@pytest.mark.parametrize("dim", [64, 128])
def test_prefix_and_own_values_far_apart(dim):
    # the join of a prefix of large values without weight and own tokens of small ones
    b = Batch(81, [90, 10, 64], heads=4, kv_heads=2, dim=dim, prefix_lens=[150], members=[0, 3])
    b.q_bits[..., 5] = 0x4100  # 8
    for gain in (2.0 ** 40, 2.0 ** -40):
        x = ru.bf16_values(workloads.random_rows(83, 300, dim))
        v = to_dev(workloads.to_bf16_bits((x * gain).astype(np.float32))).view(150, 2, dim)
        k = to_dev(workloads.random_rows(84, 300, dim, scale=0.25)).view(150, 2, dim).clone()
        k[:, :, 5] = -64.0
        fq.nvfp4_kv_append(b.cache, k, v, torch.from_numpy(b._slots(b.ptable[0], 150)).cuda())
        check(b, 1.0, "prefix %g" % gain)
