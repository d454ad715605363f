"""prompt_attention against float64, over head sizes and layouts, packed and
ragged lengths from nothing up, chunks behind a context, strides, scales and
values that are not finite."""
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


def tensor(*shape, seed=0, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 17 * len(shape) + shape[0])
    return (gain * torch.randn(shape, generator=g, device="cuda")).bfloat16()


def offsets(lens, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def inputs(q_lens, k_lens, h, hk, d, seed=0, gain=1.0):
    return (tensor(sum(q_lens), h, d, seed=seed, gain=gain), tensor(sum(k_lens), hk, d, seed=seed + 1),
            tensor(sum(k_lens), hk, d, seed=seed + 2))


def check(q, k, v, q_lens, k_lens, got, lse=None, scale=None, label="", q0=0, k0=0):
    d, rep = q.shape[2], q.shape[1] // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    for b, (m, n) in enumerate(zip(q_lens, k_lens)):
        kk, vv = (np.repeat(lu.f64(t[k0:k0 + n]), rep, 1) for t in (k, v))
        o, l, bound, lbound = lu.prompt(lu.f64(q[q0:q0 + m]), kk, vv, scale)
        lu.check(lu.f64(got[q0:q0 + m]), o, bound, "%s sequence %d (%d of %d)" % (label, b, m, n))
        if lse is not None:
            x = lu.f64(lse[q0:q0 + m])
            seen = np.isfinite(l)
            assert (x[~seen] == -math.inf).all()
            lu.check(x[seen], l[seen], lbound[seen], "%s lse %d" % (label, b))
        q0, k0 = q0 + m, k0 + n


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("h,hk", [(1, 1), (4, 4), (8, 2), (5, 1), (14, 2)])
def test_packed_lengths(d, h, hk):
    lens = [1, 0, 2, 31, 32, 33, 0, 63, 64, 65, 127, 129, 200]
    q, k, v = inputs(lens, lens, h, hk, d)
    off = offsets(lens)
    out, lse = fq.prompt_attention(q, k, v, off, lse=True)
    check(q, k, v, lens, lens, out, lse, label="packed")
    assert torch.equal(fq.prompt_attention(q, k, v, off), out)
    assert torch.equal(fq.prompt_attention(q, k, v, off, off), out)


@pytest.mark.parametrize("d", [64, 128, 192, 256])
def test_chunks_behind_a_context(d):
    q_lens, k_lens = [1, 7, 64, 1, 130, 0, 5], [1000, 71, 300, 1, 131, 40, 517]
    q, k, v = inputs(q_lens, k_lens, 6, 3, d, seed=3, gain=1.5)
    out, lse = fq.prompt_attention(q, k, v, offsets(q_lens), offsets(k_lens), lse=True)
    check(q, k, v, q_lens, k_lens, out, lse, label="chunk")


def test_more_queries_than_keys_and_no_keys():
    q_lens, k_lens = [9, 70, 3, 100, 40], [4, 0, 0, 33, 40]
    for d in (64, 128, 256):
        q, k, v = inputs(q_lens, k_lens, 4, 2, d, seed=5)
        out, lse = fq.prompt_attention(q, k, v, offsets(q_lens), offsets(k_lens), lse=True)
        check(q, k, v, q_lens, k_lens, out, lse, label="few keys")
        assert (out[:5] == 0).all() and (lse[:5] == -math.inf).all()
        out = fq.prompt_attention(q, k[:0], v[:0], offsets(q_lens), offsets([0] * 5))
        assert (out == 0).all()


@pytest.mark.parametrize("length", [255, 1025, 2500])
@pytest.mark.parametrize("d", [64, 128, 192, 256])
def test_long(d, length):
    q, k, v = inputs([length], [length], 4, 2, d, seed=7, gain=2.0)
    out, lse = fq.prompt_attention(q, k, v, offsets([length]), lse=True)
    check(q, k, v, [length], [length], out, lse, label="long")


@pytest.mark.parametrize("heads", [(40, 8), (3, 3), (32, 1), (71, 71), (130, 2)])
def test_head_counts(heads):
    lens = [50, 3, 77]
    q, k, v = inputs(lens, lens, *heads, 64, seed=9)
    check(q, k, v, lens, lens, fq.prompt_attention(q, k, v, offsets(lens)), label="heads")


def test_many_sequences():
    rng = np.random.RandomState(4)
    lens = [int(n) for n in rng.randint(0, 6, 3000)]
    q, k, v = inputs(lens, lens, 2, 1, 64, seed=11)
    out = fq.prompt_attention(q, k, v, offsets(lens))
    # every sequence of one length at once
    starts = np.concatenate([[0], np.cumsum(lens)])
    for n in range(1, 6):
        rows = torch.tensor([starts[i] + j for i, m in enumerate(lens) if m == n for j in range(n)], device="cuda")
        qs, ks, vs = (lu.f64(t[rows]).reshape(-1, n, t.shape[1], 64) for t in (q, k, v))
        got = lu.f64(out[rows]).reshape(qs.shape)
        for b in range(len(qs)):
            o, _, bound, _ = lu.prompt(qs[b], np.repeat(ks[b], 2, 1), np.repeat(vs[b], 2, 1), 1 / 8)
            lu.check(got[b], o, bound, "length %d" % n)


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("lens", [[700, 3], [0, 400, 400, 1, 257], [5, 300, 0, 128, 300, 64, 299, 1, 512, 0, 128],
                                  [(37 * i) % 90 for i in range(64)]])
def test_more_blocks_than_run_at_once(lens, d):
    # over 512 workgroups of up to 64 sequences: they go in order of length
    q, k, v = inputs(lens, lens, 130, 130, d, seed=47, gain=1.5)
    out, lse = fq.prompt_attention(q, k, v, offsets(lens), lse=True)
    some = slice(0, 130, 43)
    check(q[:, some], k[:, some], v[:, some], lens, lens, out[:, some], lse[:, some], label="by length")
    # every head, the same keys for all: each as the first
    kk, vv, qq = (t[:, :1].expand(-1, 130, -1).contiguous() for t in (k, v, q))
    out = fq.prompt_attention(qq, kk, vv, offsets(lens))
    assert torch.equal(out, out[:, :1].expand(-1, 130, -1))


def test_one_sequence_alone_is_the_same_as_packed():
    lens = [300, 17, 129]
    q, k, v = inputs(lens, lens, 8, 2, 128, seed=13)
    out = fq.prompt_attention(q, k, v, offsets(lens))
    a = 0
    for n in lens:
        check(q[a:a + n], k[a:a + n], v[a:a + n], [n], [n],
              fq.prompt_attention(q[a:a + n].contiguous(), k[a:a + n].contiguous(), v[a:a + n].contiguous(),
                                  offsets([n])), label="alone")
        a += n
    check(q, k, v, lens, lens, out, label="packed")


def test_strided_slices_of_a_projection():
    lens, h, hk, d = [90, 1, 45], 6, 2, 128
    qkv = tensor(136, h + 2 * hk + 1, d, seed=15)
    q, k, v = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:h + 2 * hk]
    out = fq.prompt_attention(q, k, v, offsets(lens))
    assert torch.equal(out, fq.prompt_attention(q.contiguous(), k.contiguous(), v.contiguous(), offsets(lens)))
    check(q, k, v, lens, lens, out, label="strided")


def test_rows_outside_the_sequences_stay():
    lens, first = [40, 0, 25], 7
    q, k, v = inputs([100], [100], 4, 2, 64, seed=17)
    out = torch.full_like(q, 3.0)
    got = fq.prompt_attention(q, k, v, offsets(lens, first), out=out)
    assert got.data_ptr() == out.data_ptr()
    assert (out[:7] == 3).all() and (out[72:] == 3).all()
    check(q, k, v, lens, lens, out, q0=7, k0=7, label="inside")


def test_offsets_are_clamped():
    # past the end, below zero and falling: every access stays inside, other sequences are right
    q, k, v = inputs([64], [64], 4, 2, 64, seed=19)
    for q_off, k_off in (([-5, 20, 900], [0, 20, 2000]), ([0, 64, 10], [0, 64, 64]),
                         ([0, 30, 64], [-9, 30, 5000]), ([70, 80, 90], [70, 80, 90])):
        a, b = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in (q_off, k_off))
        out = fq.prompt_attention(q, k, v, a, b)
        assert out.shape == q.shape
    a = torch.tensor([0, 20, 900], dtype=torch.int32, device="cuda")
    check(q, k, v, [20, 44], [20, 44], fq.prompt_attention(q, k, v, a), label="clamped end")


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.125, 1e-30, 2.0 ** 100, 2.0 ** -140, 37.0])
def test_scales(scale):
    lens = [130, 20]
    q, k, v = inputs(lens, lens, 4, 2, 64, seed=21)
    if scale > 1e20:  # one key alone has weight, or those with equal scores
        q, k = (torch.sign(t.float()).bfloat16() for t in (q, k))
        out = fq.prompt_attention(q, k, v, offsets(lens), scale=scale)
        s = (q[:20].float().transpose(0, 1) @ k[:20].float().repeat_interleave(2, 1).transpose(0, 1).transpose(1, 2))
        s = s.masked_fill(torch.ones(20, 20, device="cuda").triu(1).bool(), -math.inf)
        p = (s == s.amax(-1, keepdim=True)).float()
        want = (p / p.sum(-1, keepdim=True)) @ v[:20].float().repeat_interleave(2, 1).transpose(0, 1)
        assert torch.allclose(out[:20].float().transpose(0, 1), want, atol=0.05, rtol=0.02)
        return
    out, lse = fq.prompt_attention(q, k, v, offsets(lens), scale=scale, lse=True)
    check(q, k, v, lens, lens, out, lse, scale=scale, label="scale %g" % scale)


@pytest.mark.parametrize("gain", [2.0 ** -60, 2.0 ** 5, 2.0 ** 12])
def test_score_ranges(gain):
    # from scores that are all alike to ones of which one key alone has weight
    lens = [200]
    q, k, v = inputs(lens, lens, 2, 2, 128, seed=23, gain=gain)
    out, lse = fq.prompt_attention(q, k, v, offsets(lens), lse=True)
    check(q, k, v, lens, lens, out, lse, label="gain %g" % gain)


def test_growing_and_falling_scores():
    # the largest score comes last, first, or grows by less than the slack at every step
    n, d = 400, 64
    for slope in (0.001, 0.02, 0.05, 1.0, -0.02, -1.0):
        k = torch.zeros((n, 1, d), device="cuda")
        k[:, 0, 0] = torch.arange(n, device="cuda") * slope
        k[:, 0, 1:] = 0.01 * tensor(n, d - 1, seed=25).float()
        q = torch.ones((n, 1, d), device="cuda")
        q, k, v = q.bfloat16(), k.bfloat16(), tensor(n, 1, d, seed=27)
        out, lse = fq.prompt_attention(q, k, v, offsets([n]), scale=1.0, lse=True)
        check(q, k, v, [n], [n], out, lse, scale=1.0, label="slope %g" % slope)


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_what_a_query_does_not_see_has_no_effect(d, bad):
    lens = [70, 33, 150]
    q, k, v = inputs(lens, lens, 4, 2, d, seed=29)
    clean = fq.prompt_attention(q, k, v, offsets(lens))
    # key 40 of the last sequence, key head 1: seen by its queries from 40 on
    at = 103 + 40
    for which in ("v", "k"):
        kk, vv = k.clone(), v.clone()
        (vv if which == "v" else kk)[at, 1, 5] = bad
        out = fq.prompt_attention(q, kk, vv, offsets(lens))
        assert torch.equal(out[:at], clean[:at])
        assert torch.equal(out[at:, :2], clean[at:, :2])  # the other key head's
        seen = out[at:, 2:].float()
        if which == "v":
            if math.isinf(bad):
                assert (seen[..., 5] == bad).all()
            else:
                assert torch.isnan(seen[..., 5]).all()
            rest = torch.cat([seen[..., :5], seen[..., 6:]], -1)
            want = clean[at:, 2:].float()
            assert torch.allclose(rest, torch.cat([want[..., :5], want[..., 6:]], -1), atol=0.02, rtol=0.02)
        elif math.isnan(bad):
            assert torch.isnan(seen).all()


def test_infinite_values_behind_the_last_key():
    # rows of the tensors that belong to no sequence
    lens = [5, 60]
    q, k, v = inputs([65 + 30], [65 + 30], 4, 2, 64, seed=31)
    clean = fq.prompt_attention(q[:65].contiguous(), k[:65].contiguous(), v[:65].contiguous(), offsets(lens))
    k[65:], v[65:] = math.nan, math.inf
    out = torch.zeros_like(q)
    fq.prompt_attention(q, k, v, offsets(lens), out=out)
    assert torch.equal(out[:65], clean) and (out[65:] == 0).all()


def test_a_value_without_weight():
    # seen with a weight that underflows: infinite, or NaN as 0 times infinity is
    n, d = 80, 64
    q, k, v = torch.ones((n, 1, d)), torch.zeros((n, 1, d)), tensor(n, 1, d, seed=33)
    k[3] = -100.0
    q, k = q.cuda().bfloat16(), k.cuda().bfloat16()
    v[3, 0, 7] = math.inf
    out = fq.prompt_attention(q, k, v, offsets([n])).float()
    assert not torch.isfinite(out[3:, 0, 7]).any() and torch.isfinite(out[:3]).all()
    rest = [i for i in range(d) if i != 7]
    assert torch.isfinite(out[:, 0, rest]).all()


def test_scores_of_minus_infinity():
    # a key of -infinity takes no weight; a query that sees only such keys gives zeros
    n, d = 70, 64
    q, k, v = torch.ones((n, 1, d)).cuda().bfloat16(), tensor(n, 1, d, seed=35), tensor(n, 1, d, seed=36)
    k[0, 0, 0] = k[1, 0, 3] = k[66, 0, 3] = -math.inf
    out, lse = fq.prompt_attention(q, k, v, offsets([n]), lse=True)
    assert (out[:2] == 0).all() and (lse[:2] == -math.inf).all()
    keep = [i for i in range(n) if i not in (0, 1, 66)]
    s = (q[:, 0].double() @ k[:, 0].double().t()) * d ** -0.5
    s = s.masked_fill(torch.ones(n, n, device="cuda").triu(1).bool(), -math.inf)
    want = torch.softmax(s[2:][:, keep], 1) @ v[keep, 0].double()
    assert torch.allclose(out[2:, 0].double(), want, atol=0.03, rtol=0.02)


# contexts that are cut into parts, where queries are few (several launches)
PARTS = [(64, 8, 2, [3], [2500]), (128, 8, 1, [1], [5000]), (128, 8, 2, [40, 1, 0, 7], [3000, 2000, 1500, 5]),
         (192, 4, 4, [20], [3100]), (256, 4, 2, [5, 30], [1200, 3000]), (128, 2, 1, [64], [64 * 40]),
         (64, 6, 3, [9, 4], [0, 9000]), (256, 2, 2, [33], [1601])]


@pytest.mark.parametrize("d,h,hk,q_lens,k_lens", PARTS)
def test_few_queries_behind_long_contexts(d, h, hk, q_lens, k_lens):
    q, k, v = inputs(q_lens, k_lens, h, hk, d, seed=41, gain=1.5)
    assert fq.rollout_lib().prompt_attention_workspace_bytes(len(q), h, len(k), hk, d, len(q_lens)) > 0
    out, lse = fq.prompt_attention(q, k, v, offsets(q_lens), offsets(k_lens), lse=True)
    check(q, k, v, q_lens, k_lens, out, lse, label="parts")
    assert torch.equal(fq.prompt_attention(q, k, v, offsets(q_lens), offsets(k_lens)), out)
    # as one call of many sequences, which are not cut, gives it
    both = (torch.cat([q] * 70), torch.cat([k] * 70), torch.cat([v] * 70))
    off = offsets(q_lens * 70), offsets(k_lens * 70)
    whole = fq.prompt_attention(*both, *off)
    check(q, k, v, q_lens, k_lens, whole[:len(q)], label="whole")
    assert torch.equal(whole[:len(q)], whole[-len(q):])


def test_parts_with_values_that_are_not_finite():
    q_lens, k_lens = [12, 3], [2000, 1800]
    q, k, v = inputs(q_lens, k_lens, 4, 2, 128, seed=43)
    args = offsets(q_lens), offsets(k_lens)
    clean = fq.prompt_attention(q, k, v, *args)
    vv = v.clone()
    vv[100, 0, 3] = math.inf            # seen by every query of the first sequence
    vv[1995, 1, 9] = -math.inf          # by its last five (12 of 2000: from 1988 on)
    vv[2000 + 1799, 0, 1] = math.nan    # by the last query of the second
    vv[2000, 1, 127] = math.nan
    out = fq.prompt_attention(q, k, vv, *args).float()
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[:12, :2, 3] = bad[7:12, 2:, 9] = bad[14, :2, 1] = bad[12:, 2:, 127] = True
    assert not torch.isfinite(out[bad]).any()
    assert torch.equal(out[~bad], clean.float()[~bad])
    # rows of no sequence stay, also behind a join
    big = torch.full((len(q) + 9, 4, 128), 3.0, device="cuda").bfloat16()
    qq = torch.cat([q[:4], q, q[:5]])
    fq.prompt_attention(qq, k, v, args[0] + 4, args[1], out=big)
    assert torch.equal(big[4:4 + len(q)], clean) and (big[:4] == 3).all() and (big[4 + len(q):] == 3).all()


def test_workspaces():
    q, k, v = inputs([4], [4000], 4, 2, 128, seed=45)
    args = (q, k, v, offsets([4]), offsets([4000]))
    need = fq.rollout_lib().prompt_attention_workspace_bytes(4, 4, 4000, 2, 128, 1)
    out = fq.prompt_attention(*args)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")  # contents are ignored
    assert torch.equal(fq.prompt_attention(*args, workspace=ws), out)
    with pytest.raises(fq.Fp4qError):
        fq.prompt_attention(*args, workspace=ws[:need - 1])


def test_keys_past_32_bit_offsets():
    # rows of keys and values far apart: the last begins beyond 2^31 elements
    n, stride = 300, 1 << 23
    big = torch.empty((n - 1) * stride + 256, dtype=torch.bfloat16, device="cuda")
    k, v = (big.as_strided((n, 2, 64), (stride, 64, 1), storage_offset=s) for s in (0, 128))
    ks, vs = tensor(n, 2, 64, seed=37), tensor(n, 2, 64, seed=38)
    k.copy_(ks)
    v.copy_(vs)
    q = tensor(n, 4, 64, seed=39)
    out = fq.prompt_attention(q, k, v, offsets([n]))
    assert torch.equal(out, fq.prompt_attention(q, ks, vs, offsets([n])))
