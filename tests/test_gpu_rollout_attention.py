"""nvfp4_kv_attention on the GPU against attention in float64 over the cache's
exact values, with the error bound of rolloututil.attention.  Every place
that no sequence uses holds NaN scales, so that nothing masked can leak."""
import math

import numpy as np
import pytest
import torch

import fp4_block_quantization_amd as fq
import rolloututil as ru
import workloads
from gpuutil import Guards, bits_of, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.rollout_lib()


def poisoned(pages, page, heads, dim):
    c = fq.nvfp4_kv_cache(pages, page, heads, dim)
    for i in (0, 3):
        c[i].fill_(0xFF)
        c[i + 1].fill_(0x7F)           # an E4M3 NaN
        c[i + 2].fill_(float("nan"))
    return c


class Batch:
    """A batch of sequences with their pages, queries and prefixes."""

    def __init__(self, seed, lens, tokens=1, heads=4, kv_heads=2, dim=64, page=16, prefix_lens=(),
                 members=(), max_pages=None, q_gain=1.0, gain_sigma=0.7):
        rng = np.random.default_rng(seed)
        self.lens, self.tokens, self.heads, self.kv_heads = list(lens), tokens, heads, kv_heads
        self.dim, self.page, self.prefix_lens, self.members = dim, page, prefix_lens, members
        batch = len(self.lens)
        per = max_pages or max(1, -(-max(self.lens, default=1) // page))
        pper = -(-max(prefix_lens, default=0) // page)
        groups = len(prefix_lens)
        pages = batch * per + groups * pper + 1
        self.cache = poisoned(pages, page, kv_heads, dim)
        ids = rng.permutation(pages)[:pages - 1].astype(np.int32)
        self.table = ids[:batch * per].reshape(batch, per).copy()
        self.ptable = ids[batch * per:].reshape(groups, pper).copy() if groups else None
        slots = [self._slots(self.table[b], n) for b, n in enumerate(self.lens)]
        slots += [self._slots(self.ptable[g], n) for g, n in enumerate(prefix_lens)]
        slots = np.concatenate(slots).astype(np.int64)
        kb, vb = (workloads.random_rows(seed * 2 + i, max(1, len(slots)) * kv_heads, dim,
                                        row_gain_sigma=gain_sigma) for i in (1, 2))
        if len(slots):
            fq.nvfp4_kv_append(self.cache, *(to_dev(b).view(len(slots), kv_heads, dim)
                                             for b in (kb, vb)), torch.from_numpy(slots).cuda())
        # pages that a sequence's end leaves unused in its table: ids outside the cache
        for b, n in enumerate(self.lens):
            self.table[b, -(-n // page):] = (1 << 30) if b % 2 else -7
        q = workloads.random_rows(seed * 2 + 9, batch * tokens * heads, dim)
        q = workloads.to_bf16_bits((ru.bf16_values(q) * q_gain).astype(np.float32))
        self.q_bits = q.reshape(batch, tokens, heads, dim)

    def _slots(self, row, n):
        at = np.arange(n)
        return row[at // self.page].astype(np.int64) * self.page + at % self.page

    def prefix(self):
        if self.ptable is None:
            return None
        off = np.asarray(self.members, np.int32)
        return tuple(torch.from_numpy(np.asarray(a, np.int32)).cuda()
                     for a in (self.ptable, self.prefix_lens, off))

    def run(self, **kw):
        q = to_dev(self.q_bits.reshape(-1, self.dim)).view(self.q_bits.shape)
        return fq.nvfp4_kv_attention(q, self.cache, torch.from_numpy(self.table).cuda(),
                                     torch.tensor(self.lens, dtype=torch.int32, device="cuda"),
                                     prefix=self.prefix(), **kw)

    def _values(self, row, n):
        slots = self._slots(row, n)
        out = []
        for i in (0, 3):
            codes, scales, ts = self.host[i:i + 3]
            if i:
                scales = scales.swapaxes(2, 3)
            pg, at = slots // self.page, slots % self.page
            out.append(ru.nv_values(codes[pg, :, at], scales[pg, :, at], ts[pg, :, at]))
        return out

    def check(self, scale=None, label="", **kw):
        gu = Guards()
        out = gu.empty(self.q_bits.shape, torch.bfloat16)
        out.view(torch.uint8).fill_(0xFF)
        got, lse = self.run(scale=scale, out=out, lse=True, **kw)
        gu.check(label)
        got, lse = got.float().cpu().numpy(), lse.cpu().numpy()
        self.host = [t.cpu().numpy() for t in self.cache]
        scale = 1.0 / math.sqrt(self.dim) if scale is None else scale
        rep = self.heads // self.kv_heads
        for b, n in enumerate(self.lens):
            k, v = self._values(self.table[b], n)
            before = 0
            for g, pn in enumerate(self.prefix_lens):
                if self.members[g] <= b < self.members[g + 1]:
                    pk, pv = self._values(self.ptable[g], pn)
                    k, v, before = np.concatenate([pk, k]), np.concatenate([pv, v]), pn
            k, v = (np.repeat(t, rep, 1) for t in (k, v))
            for i in range(self.tokens):
                m = before + max(0, n - self.tokens + 1 + i)
                q = ru.bf16_values(self.q_bits[b, i])
                r = ru.attention(q, k[:m], v[:m], scale)
                where = "%s sequence %d (%d of %d keys) query %d" % (label, b, m, before + n, i)
                ru.check(got[b, i], r[0], r[2], where)
                if m == 0:
                    assert np.isneginf(lse[b, i]).all(), where
                else:
                    ru.check(lse[b, i], r[1], r[3] + 2.0 ** -20 * np.abs(r[1]), where + " lse")


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("page", [16, 48, 64, 128])
def test_lengths(dim, page):
    lens = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 200, 255, 257, 391]
    Batch(dim + page, lens, dim=dim, page=page).check(label="d=%d page=%d" % (dim, page))


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (2, 2), (8, 1), (5, 5), (15, 3), (16, 1),
                                            (24, 2), (34, 2), (71, 1)])
def test_head_layouts(heads, kv_heads):
    Batch(heads * 7 + kv_heads, [70, 5, 130], heads=heads, kv_heads=kv_heads,
          dim=128).check(label="%d/%d" % (heads, kv_heads))


@pytest.mark.parametrize("tokens", [2, 3, 5, 16, 33])
def test_several_queries_per_sequence(tokens):
    # lengths below the query count leave the first queries nothing to see
    Batch(tokens, [0, 1, tokens - 1, tokens, tokens + 1, 80, 150], tokens=tokens, heads=6,
          kv_heads=2).check(label="%d queries" % tokens)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("prefix_lens,members,lens", [
    ([100], [0, 3], [5, 0, 70]),
    ([64, 0, 201], [0, 2, 3, 7], [1, 64, 0, 9, 130, 2, 33]),
    ([300, 17], [1, 4, 5], [8, 0, 0, 40, 3, 90]),          # the first and last in no group
    ([129, 50, 70], [0, 0, 5, 5], [3, 3, 3, 3, 3]),        # groups of nobody
    ([500], [0, 40], [i % 7 for i in range(40)]),
])
def test_shared_prefix(prefix_lens, members, lens, dim):
    for tokens in (1, 2):
        Batch(sum(lens) + dim, lens, tokens=tokens, heads=8, kv_heads=2, dim=dim,
              prefix_lens=prefix_lens, members=members).check(label="prefix t=%d" % tokens)


def test_long_contexts_in_many_parts():
    Batch(3, [3000, 1, 2049, 777], heads=8, kv_heads=1, dim=128, page=64).check(label="long")
    Batch(4, [40, 7], heads=4, kv_heads=1, dim=64, prefix_lens=[5000], members=[0, 2],
          page=32).check(label="long prefix")
    # a table much wider than the sequences
    Batch(5, [100, 3], heads=4, kv_heads=2, dim=64, max_pages=600).check(label="wide table")


@pytest.mark.parametrize("dim,heads,kv_heads,tokens", [(64, 4, 2, 1), (128, 8, 2, 1), (192, 6, 2, 2),
                                                       (256, 2, 1, 1), (64, 20, 2, 3),
                                                       (128, 40, 1, 1), (256, 9, 1, 3)])
def test_wide_tables(dim, heads, kv_heads, tokens):
    # tables with room for more than 2048 tokens: contexts laid end to end and cut into pieces,
    # with cuts inside short and long ones, and empty ones between them
    lens = [0, 700, 1, 64, 65, 0, 0, 1500, 63, 129, 2100, 5, 320]
    Batch(dim + heads, lens, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, page=32,
          max_pages=70).check(label="wide %d" % dim)


def test_many_sequences():
    # more sequences (and groups) than one round of a workgroup's threads
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 40, 300)
    Batch(21, lens, heads=2, kv_heads=1, dim=64, max_pages=130).check(label="many")
    members = np.minimum(np.arange(0, 291), 290)
    Batch(22, lens, heads=2, kv_heads=1, dim=64, prefix_lens=rng.integers(0, 70, 290),
          members=members).check(label="many groups")


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("max_pages", [4, 140])
def test_many_sequences_with_many_rows(dim, max_pages):
    # enough items that workgroups take two row tiles of 16 (up to heads of 128): 28 rows
    # each, one of them short; whole contexts, and contexts cut into parts
    rng = np.random.default_rng(dim)
    lens = rng.integers(0, 65, 90)
    lens[:4] = 0, 1, 6, 7
    Batch(31, lens, tokens=7, heads=12, kv_heads=3, dim=dim, max_pages=max_pages).check(
        label="%d pages" % max_pages)


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_many_short_contexts(dim):
    # more items than eight wavefronts each would fill the chip with at once
    rng = np.random.default_rng(dim + 1)
    lens = rng.integers(0, 300, 90)
    lens[:5] = 0, 1, 63, 64, 65
    Batch(33, lens, heads=12, kv_heads=6, dim=dim).check(label="many short")


@pytest.mark.parametrize("tokens", [1, 7])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_many_sequences_in_parts(dim, tokens):
    # many items whose tables have room for more than 4096 tokens: contexts cut into parts, one
    # row tile or two, the part found by all threads of a workgroup
    rng = np.random.default_rng(dim + tokens)
    lens = rng.integers(0, 200, 90)
    lens[:5] = 0, 1, 6, 1300, 64
    Batch(34, lens, tokens=tokens, heads=12, kv_heads=3, dim=dim, max_pages=260).check(
        label="in parts")


@pytest.mark.parametrize("dim", [64, 128, 192])
def test_shared_prefix_of_many_rows(dim):
    # groups of more than 256 rows on average, one of them small, one with an odd count
    lens = [i % 5 for i in range(23)]
    Batch(32, lens, tokens=3, heads=32, kv_heads=1, dim=dim, prefix_lens=[150, 333],
          members=[0, 2, 23]).check(label="rows")


@pytest.mark.parametrize("gain,scale", [(1.0, 0.0), (1.0, -0.3), (30.0, 1.0), (2.0 ** 60, 2.0 ** -60),
                                        (2.0 ** -70, 2.0 ** 70), (1e-3, 1.0)])
def test_scales_of_the_scores(gain, scale):
    Batch(11, [100, 1, 33], dim=128, q_gain=gain).check(scale=scale, label="%g %g" % (gain, scale))


@pytest.mark.parametrize("sigma", [3.0, 8.0])
def test_token_scales_far_apart(sigma):
    # token scales over e^(+-3 sigma): rows may rest on tokens whose values are tiny
    Batch(12, [300, 64, 90], dim=64, gain_sigma=sigma, q_gain=1e-2).check(label="sigma %g" % sigma)


def test_zero_rows_of_the_cache():
    b = Batch(13, [50, 1, 3], dim=64)
    zero = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    slots = np.concatenate([b._slots(b.table[0], 50)[[0, 7]], b._slots(b.table[1], 1)])
    fq.nvfp4_kv_append(b.cache, zero, zero, torch.from_numpy(slots).cuda())
    b.check(label="zero rows")


def test_a_nan_query_stays_in_its_row():
    b = Batch(14, [90, 40], heads=4, kv_heads=1, dim=64)
    b.q_bits[0, 0, 1, 3] = 0x7FC0
    got = b.run().float().cpu().numpy()
    assert np.isnan(got[0, 0, 1]).all()
    got[0, 0, 1] = 0
    assert np.isfinite(got).all()
    b.q_bits[0, 0, 1] = b.q_bits[0, 0, 0]
    clean = b.run().float().cpu().numpy()
    keep = np.ones(got.shape[:3], bool)
    keep[0, 0, 1] = False
    assert np.array_equal(got[keep], clean[keep])


def test_strided_queries_streams_and_lengths_past_the_table():
    b = Batch(15, [30, 64, 9], tokens=2, heads=4, kv_heads=2, dim=64)
    want = b.run()
    fused = torch.zeros((3, 2, 8, 64), dtype=torch.bfloat16, device="cuda")
    fused[:, :, 2:6] = to_dev(b.q_bits.reshape(-1, 64)).view(b.q_bits.shape)
    table = torch.from_numpy(b.table).cuda()
    lens = torch.tensor([30, 1 << 30, 9], dtype=torch.int32, device="cuda")  # clamped to 64
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = fq.nvfp4_kv_attention(fused[:, :, 2:6], b.cache, table, lens)
    side.synchronize()
    assert np.array_equal(bits_of(got), bits_of(want))
    neg = torch.tensor([-4, 64, 9], dtype=torch.int32, device="cuda")
    assert not fq.nvfp4_kv_attention(fused[:, :, 2:6], b.cache, table, neg)[0].any()


def test_three_dimensional_queries_and_refusals():
    b = Batch(16, [30, 64], heads=4, kv_heads=2, dim=64)
    q = to_dev(b.q_bits.reshape(-1, 64)).view(2, 4, 64)
    table = torch.from_numpy(b.table).cuda()
    lens = torch.tensor(b.lens, dtype=torch.int32, device="cuda")
    assert np.array_equal(bits_of(fq.nvfp4_kv_attention(q, b.cache, table, lens)).ravel(),
                          bits_of(b.run()).ravel())
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    good = dict(q=q, cache=b.cache, page_table=table, seq_lens=lens)
    for kw in (dict(q=q.float()), dict(q=q.transpose(1, 2)), dict(q=q[:, :3]), dict(q=q[0]),
               dict(page_table=table.long()), dict(page_table=table[:1]), dict(seq_lens=lens[:1]),
               dict(seq_lens=lens.long()), dict(prefix=(i32(0, 3), i32(0), i32(1))),
               dict(prefix=(i32(1, 3), i32(2), i32(2))), dict(prefix=(i32(1, 3), i32(1), i32(1))),
               dict(out=torch.empty_like(q).float()), dict(scale=float("inf")),
               dict(q=q.cpu()), dict(cache=b.cache[:4])):
        with pytest.raises(fq.Fp4qError):
            fq.nvfp4_kv_attention(**{**good, **kw})
    assert fq.nvfp4_kv_attention(q[:0], b.cache, table[:0], lens[:0]).shape == (0, 4, 64)
