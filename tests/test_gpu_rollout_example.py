"""The rollout example: its operators' results, call by call, against float64
on the CPU, and its captured graph, replayed with eager work between the
replays, against eager steps bit for bit."""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

import fp4_block_quantization_amd as fq
import rolloututil as ru

pytestmark = pytest.mark.gpu
SIZES = dict(hidden=256, heads=6, kv_heads=2, dim=64, experts=5, ffn=96)


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    path = os.path.join(root, "examples", "rollout_decode.py")
    spec = importlib.util.spec_from_file_location("rollout_decode", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def start(example, steps=24):
    torch.manual_seed(3)
    layer = example.Layer(**SIZES)
    prompts = torch.randn((3, 37, SIZES["hidden"]), device="cuda").bfloat16()
    return example.Rollout(layer, prompts, samples=2, steps=steps, page=16)


def f64(t):
    return t.double().cpu().numpy()


def check_product(x, w, y, label):
    want, bound = ru.linear_bound(f64(x), w, out_bf16=True)
    ru.check(f64(y), want, bound, label)


def check_step(example, roll, step, keys, values, label):
    """keys, values: float64 [batch, tokens, kv_heads, d] that each sequence's
    queries see, the last of them the queries' own."""
    layer = roll.layer
    batch, tokens, hidden = step.x.shape
    qkv, o = (ru.nv_values(*(t.cpu().numpy() for t in w)) for w in (layer.qkv, layer.o))
    check_product(example.norm(step.x).view(-1, hidden), qkv, step.qkv, label + " qkv")
    q = f64(step.qkv).reshape(batch, tokens, -1, layer.dim)[:, :, :layer.heads]
    rep = layer.heads // layer.kv_heads
    for b in range(batch):
        k, v = (np.repeat(t[b], rep, 1) for t in (keys, values))
        for i in range(tokens):
            seen = k.shape[0] - tokens + 1 + i
            want, _, bound, _ = ru.attention(q[b, i], k[:seen], v[:seen], 1 / math.sqrt(layer.dim))
            ru.check(f64(step.attended[b, i]), want, bound, "%s attention %d %d" % (label, b, i))
    projected = fq.nvfp4_linear(step.attended.view(batch * tokens, -1), *layer.o)
    check_product(step.attended.view(batch * tokens, -1), o, projected, label + " output")
    assert torch.equal(projected + step.x.view(-1, hidden), step.mixed), label
    order, off = roll._route(batch * tokens)
    off = off.tolist()
    for x, w, y in ((step.routed, layer.up, step.up), (step.act, layer.down, step.down)):
        for e in range(layer.experts):
            rows = slice(off[e], off[e + 1])
            if off[e] < off[e + 1]:
                check_product(x[rows], ru.mx_values(*(t[e].cpu().numpy() for t in w)), y[rows],
                              "%s expert %d" % (label, e))


def cached(roll, slots):
    """float64 [.., kv_heads, d] keys and values of slots, from the cache's bytes."""
    page, slots = roll.page, slots.cpu().numpy()
    pg, at = slots // page, slots % page
    c = [t.cpu().numpy() for t in roll.cache]
    return [ru.nv_values(codes[pg, :, at], scales[pg, :, at], ts[pg, :, at])
            for codes, scales, ts in ((c[0], c[1], c[2]), (c[3], c[4].swapaxes(2, 3), c[5]))]


def test_every_operator_of_prefill_and_decode(example):
    roll = start(example)
    n, length = 3, 37
    place = torch.arange(length, device="cuda")
    slots = roll.prompt_pages.long()[:, place // 16] * 16 + place % 16
    prompt_kv = cached(roll, slots)
    check_step(example, roll, roll.prefill, *prompt_kv, "prefill")
    kept = []
    for i in range(19):  # past a page
        at = roll.slots(torch.full_like(roll.lens, i))
        # the samples' state is overwritten by the step
        kept.append((roll.x.clone(), roll.decode(), at))
    for i in (0, 1, 16, 18):
        x, step, _ = kept[i]
        own = cached(roll, torch.stack([at for _, _, at in kept[:i + 1]], 1))
        seen = [np.concatenate([np.repeat(p, 2, 0), t], 1) for p, t in zip(prompt_kv, own)]
        check_step(example, roll, step._replace(x=x), *seen, "step %d" % i)
    # the cache holds the quantized rows of the projections, and reads them back
    k, v = fq.nvfp4_kv_read(roll.cache, kept[4][2])
    rows = kept[4][1].qkv.view(6, -1, 64)
    for got, src in ((k, rows[:, 6:8]), (v, rows[:, 8:])):
        want = fq.nvfp4_quantize(src.reshape(-1, 64), dequant=True)[3]
        assert torch.equal(got.reshape(-1, 64).view(torch.int16), want.view(torch.int16))


def test_graph_replays_equal_eager_steps(example):
    roll = start(example)
    want = []
    for _ in range(20):
        s = roll.decode()
        want.append([t.clone() for t in s[1:]])
    cache = [t.clone() for t in roll.cache]
    graph, step = roll.capture()
    for t in roll.cache:
        t.view(torch.uint8)[roll.prompt_pages.numel():].fill_(0x33)  # every sample's page
    roll.reset()
    for i in range(20):
        graph.replay()
        if i % 3 == 0:  # eager calls with workspaces of their own, and a wait
            fq.nvfp4_linear(step.attended.view(6, -1), *roll.layer.o)
            fq.nvfp4_kv_attention(torch.zeros((6, 6, 64), dtype=torch.bfloat16, device="cuda"),
                                  roll.cache, roll.pages, roll.lens, prefix=roll.prefix)
            torch.cuda.synchronize()
        for name, got, exp in zip(step._fields[1:], step[1:], want[i]):
            assert torch.equal(got.view(torch.int16), exp.view(torch.int16)), (i, name)
    slots = torch.cat([roll.slots(torch.full_like(roll.lens, i)) for i in range(20)])
    for got, exp in zip(fq.nvfp4_kv_read(roll.cache, slots),
                        fq.nvfp4_kv_read(fq.NvFp4KvCache(*cache), slots)):
        assert torch.equal(got.view(torch.int16), exp.view(torch.int16))
