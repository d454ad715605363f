"""nvfp4_kv_attention where scores leave the ordinary range: score factors
and queries so small that their product leaves FP32, keys and queries whose
magnitudes make up for each other, and scores whose spacing in FP32 is more
than one."""
import numpy as np
import pytest
import torch

import fp4_block_quantization_amd as fq
import rolloututil as ru
import workloads
from gpuutil import to_dev
from test_gpu_rollout_attention import Batch

pytestmark = pytest.mark.gpu

LENS = [100, 1, 33, 0, 64, 65]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.rollout_lib()


def scaled_bits(bits, gain):
    return workloads.to_bf16_bits((ru.bf16_values(bits) * gain).astype(np.float32))


def rewrite_keys(b, gain):
    """New keys times gain and new values in the slots of every sequence."""
    slots = np.concatenate([b._slots(b.table[i], n) for i, n in enumerate(b.lens)]).astype(np.int64)
    k, v = (workloads.random_rows(77 + i, len(slots) * b.kv_heads, b.dim) for i in (0, 1))
    k, v = (to_dev(t).view(len(slots), b.kv_heads, b.dim) for t in (scaled_bits(k, gain), v))
    fq.nvfp4_kv_append(b.cache, k, v, torch.from_numpy(slots).cuda())


@pytest.mark.parametrize("tokens", [1, 3])
@pytest.mark.parametrize("gain,scale", [
    (1.0, 1e-42), (1.0, -1e-42), (1.0, 2.0 ** -149), (2.0 ** -126, 2.0 ** -11),
    (2.0 ** -131, 2.0 ** -5), (2.0 ** -120, 2.0 ** -120), (2.0 ** 100, 1e-42)])
def test_vanishing_factors(gain, scale, tokens):
    # the scores all but vanish: the mean of what is seen, and nothing of what is masked
    Batch(41, LENS, tokens=tokens, dim=128, q_gain=gain).check(scale=scale,
                                                               label="%g %g" % (gain, scale))


@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("q_gain,k_gain,scale", [
    (2.0 ** -100, 2.0 ** 100, 0.1), (2.0 ** -60, 2.0 ** 110, 2.0 ** -50),
    (2.0 ** 100, 2.0 ** -100, 0.1), (2.0 ** 40, 2.0 ** -110, 2.0 ** 70),
    (2.0 ** -120, 2.0 ** 118, 1.0)])
def test_queries_and_keys_that_make_up_for_each_other(q_gain, k_gain, scale, dim):
    b = Batch(42, LENS, dim=dim, q_gain=q_gain)
    rewrite_keys(b, k_gain)
    b.check(scale=scale, label="%g %g %g" % (q_gain, k_gain, scale))


def test_queries_far_apart():
    # heads of one sequence, side by side in a matrix instruction, from 2^-110 to 2^20
    b = Batch(43, LENS, heads=8, kv_heads=2, dim=128)
    for h in range(8):
        b.q_bits[:, :, h] = scaled_bits(b.q_bits[:, :, h].reshape(-1, 128),
                                        2.0 ** (20 - 130 * h // 7)).reshape(len(LENS), 1, 128)
    b.check(scale=2.0 ** -20, label="apart")


@pytest.mark.parametrize("tokens", [1, 2])
@pytest.mark.parametrize("scale", [2.0 ** 18, 2.0 ** 30, -2.0 ** 45, 2.0 ** 100])
def test_scores_far_beyond_one(scale, tokens):
    # FP32 tells such scores apart by more than one: only the largest has any weight.  Keys of
    # small whole numbers have products that are exact, whatever is summed first
    b = Batch(44, LENS, tokens=tokens, heads=4, kv_heads=2, dim=64)
    rng = np.random.default_rng(3)
    slots = np.concatenate([b._slots(b.table[i], n) for i, n in enumerate(b.lens)]).astype(np.int64)
    k = rng.integers(-3, 4, (len(slots), 2, 64)).astype(np.float32)
    k[:, :, ::16] = 6.0  # every block's scale is one, or two thirds
    v = workloads.random_rows(5, len(slots) * 2, 64)
    fq.nvfp4_kv_append(b.cache, torch.from_numpy(k).bfloat16().cuda(),
                       to_dev(v).view(len(slots), 2, 64), torch.from_numpy(slots).cuda(),
                       four_over_six=False)
    q = rng.integers(-2, 3, b.q_bits.shape).astype(np.float32)
    b.q_bits = workloads.to_bf16_bits(q.reshape(-1, 64)).reshape(b.q_bits.shape)
    got, lse = b.run(scale=scale, lse=True)
    got, lse = got.float().cpu().numpy(), lse.cpu().numpy()
    b.host = [t.cpu().numpy() for t in b.cache]
    for i, n in enumerate(b.lens):
        kk, vv = b._values(b.table[i], n)
        for t in range(tokens):
            m = max(0, n - tokens + 1 + t)
            for h in range(4):
                where = "sequence %d query %d head %d" % (i, t, h)
                if m == 0:
                    assert not got[i, t, h].any() and np.isneginf(lse[i, t, h]), where
                    continue
                s = (kk[:m, h // 2] @ q[i, t, h].astype(np.float64)) * np.sign(scale)
                # the token scale's own rounding may order equal products: leave near ties out
                order = np.sort(s)
                near = s >= order[-1] - 2.0 ** -18 * np.abs(s).max()
                assert np.isfinite(got[i, t, h]).all() and np.isfinite(lse[i, t, h]), where
                np.testing.assert_allclose(lse[i, t, h], order[-1] * abs(scale), rtol=2.0 ** -17,
                                           atol=1.0, err_msg=where)
                if near.sum() == 1:
                    want = vv[np.argmax(s), h // 2]
                    assert (np.abs(got[i, t, h] - want)
                            <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * np.abs(vv).max()).all(), where
