"""The mixture-of-experts example: every operator's result of its prompts and
decoding, call by call, against float64 on the CPU, and its captured graph,
padded, replayed with eager work between the replays, against eager steps."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import fp4_block_quantization_amd as fq
import layerutil as lu
import rolloututil as ru

pytestmark = pytest.mark.gpu
SIZES = dict(hidden=256, heads=6, kv_heads=2, dim=64, experts=16, groups=4, top_groups=2, top_k=3, ffn=96)


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("rollout_moe", os.path.join(root, "examples", "rollout_moe.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def product(x, w, y, label):
    want, bound = ru.linear_bound(lu.f64(x), w, out_bf16=True)
    lu.check(lu.f64(y), want, bound, label)


def check_layer(example, layer, step, positions, tokens, label):
    """Everything of a step but its attention; tokens: how many are no padding."""
    weights = lambda w: ru.nv_values(*(t.cpu().numpy() for t in w))
    n = tokens
    product(example.norm(step.x), weights(layer.qkv), step.qkv.reshape(len(step.x), -1), label + " qkv")
    rows = lu.f64(step.qkv)
    h, hk = layer.heads, layer.kv_heads
    for got, x in ((step.q, rows[:, :h]), (step.k, rows[:, h:h + hk])):
        want, bound = lu.rotary(x, positions.cpu().numpy(), lu.f64(layer.frequencies), layer.amplitude, False, False, True)
        lu.check(lu.f64(got), want, bound, label + " rotary")
    assert torch.equal(step.v, step.qkv[:, h + hk:])
    w, e = lu.route(lu.f64(step.logits)[:n], layer.top_k, lu.f64(layer.bias), "sigmoid", layer.groups, layer.top_groups,
                    True, 1.0)
    assert np.array_equal(step.experts[:n].cpu().numpy(), e), label
    assert np.allclose(step.weights[:n].cpu().numpy(), w, rtol=1e-5)
    assert (step.experts[n:] == -1).all() and (step.weights[n:] == 0).all()
    off, place = lu.dispatch(step.experts.cpu().numpy(), layer.experts)
    assert np.array_equal(step.offsets.cpu().numpy(), off) and np.array_equal(step.place.cpu().numpy(), place)
    token, choice = np.nonzero(place >= 0)
    order = torch.from_numpy(place[token, choice]).cuda()
    assert torch.equal(step.rows[order], step.normed[torch.from_numpy(token).cuda()])
    for x, wq, y in ((step.rows, layer.up, step.up), (step.act, layer.down, step.down)):
        for i in range(layer.experts):
            if off[i] < off[i + 1]:
                product(x[off[i]:off[i + 1]], weights([t[i] for t in wq]), y[off[i]:off[i + 1]], "%s expert %d" % (label, i))
    y, p = lu.f64(step.down), place
    terms = np.where((p >= 0)[..., None], lu.f64(step.weights)[..., None] * y[np.maximum(p, 0)], 0.0)
    want, mag = lu.f64(step.mixed) + terms.sum(1), np.abs(lu.f64(step.mixed)) + np.abs(terms).sum(1)
    bound = (2 * layer.top_k + 1) * lu.FP32 * mag
    lu.check(lu.f64(step.out), want, bound + lu.BF16 * (np.abs(want) + bound), label + " sum")


def repeat(t, layer):
    return np.repeat(lu.f64(t), layer.heads // layer.kv_heads, 1)


def cached(roll, slots):
    """float64 [tokens, kv_heads, d] keys and values of slots, from the cache's bytes."""
    slots = slots.cpu().numpy()
    pg, at = slots // roll.page, slots % roll.page
    c = [t.cpu().numpy() for t in roll.cache]
    return [ru.nv_values(codes[pg, :, at], scales[pg, :, at], ts[pg, :, at])
            for codes, scales, ts in ((c[0], c[1], c[2]), (c[3], c[4].swapaxes(2, 3), c[5]))]


def test_prompts_in_chunks_and_decode(example):
    torch.manual_seed(5)
    layer = example.Layer(**SIZES)
    lens = [70, 1, 33]
    roll = example.Rollout(layer, lens, 100, room=5, page=16)
    prompts = [torch.randn((n, SIZES["hidden"]), device="cuda").bfloat16() for n in lens]
    steps = roll.prefill(prompts, 40)
    assert len(steps) == 2 and roll.lens.tolist() == lens + [0, 0]
    scale = layer.dim ** -0.5
    done = [0, 0, 0]
    for c, step in enumerate(steps):
        new = [min(40, n - d) for n, d in zip(lens, done)]
        pos = torch.cat([torch.arange(d, d + m) for d, m in zip(done, new)])
        check_layer(example, layer, step, pos, len(step.x), "chunk %d" % c)
        a = 0
        for i, (d, m) in enumerate(zip(done, new)):
            if c == 0:
                k, v = step.k[a:a + m], step.v[a:a + m]
            else:
                k, v = fq.nvfp4_kv_read(roll.cache, roll.slots(torch.full((d + m,), i, device="cuda"),
                                                               torch.arange(d + m, device="cuda")))
            o, _, bound, _ = lu.prompt(lu.f64(step.q[a:a + m]), repeat(k, layer), repeat(v, layer), scale)
            lu.check(lu.f64(step.attended[a:a + m]), o, bound, "chunk %d sequence %d" % (c, i))
            a += m
        done = [d + m for d, m in zip(done, new)]
    # the cache holds the turned keys, as quantized rows
    slots = roll.slots(torch.full((30,), 0, device="cuda"), torch.arange(40, 70, device="cuda"))
    k, v = fq.nvfp4_kv_read(roll.cache, slots)
    for got, src in ((k, steps[1].k[:30]), (v, steps[1].v[:30])):
        want = fq.nvfp4_quantize(src.reshape(-1, layer.dim).contiguous(), dequant=True)[3]
        assert torch.equal(got.reshape(-1, layer.dim), want)
    for i in range(3):
        at = roll.lens.clone()
        x = roll.x.clone()
        step = roll.decode()
        check_layer(example, layer, step._replace(x=x), at, 3, "decode %d" % i)
        assert roll.lens.tolist() == [n + i + 1 for n in lens] + [0, 0]
        for s in range(3):
            n = lens[s] + i + 1
            k, v = cached(roll, roll.slots(torch.full((n,), s, device="cuda"), torch.arange(n, device="cuda")))
            rep = layer.heads // layer.kv_heads
            o, _, bound, _ = ru.attention(lu.f64(step.q[s]), np.repeat(k, rep, 1), np.repeat(v, rep, 1), scale)
            lu.check(lu.f64(step.attended[s]), o, bound, "decode %d sequence %d" % (i, s))
        assert (step.attended[3:] == 0).all()


def test_graph_replays_equal_eager_steps(example):
    def start():
        torch.manual_seed(6)
        layer = example.Layer(**SIZES)
        roll = example.Rollout(layer, [20, 9, 31], 60, room=4, page=16)
        roll.prefill([torch.randn((n, SIZES["hidden"]), device="cuda").bfloat16() for n in (20, 9, 31)], 64)
        return roll

    roll = start()
    want = []
    for _ in range(17):
        s = roll.decode()
        want.append([t[:3].clone() for t in (s.q, s.attended, s.weights, s.experts, s.place, s.out)])
    roll = start()
    graph, step = roll.capture()
    for i in range(17):
        graph.replay()
        if i % 3 == 0:
            fq.moe_dispatch(step.normed, step.experts, 16)
            torch.cuda.synchronize()
        got = (step.q, step.attended, step.weights, step.experts, step.place, step.out)
        for name, a, b in zip("q attended weights experts place out".split(), got, want[i]):
            assert torch.equal(a[:3], b), (i, name)
