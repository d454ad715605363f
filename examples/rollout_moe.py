"""A mixture-of-experts layer of a rollout engine, prompts and decoding, all on
the framework's operators.

  prompts    of mixed length, packed: fused QKV product -> rotary positions ->
             cache write -> attention over the prompts in BF16; long ones in
             chunks, each behind what the cache holds, read back
  decode     one token of every sequence in a captured graph, padded to a
             fixed batch: the same, with attention over the NVFP4 cache
  experts    scores -> the best of each token -> rows by expert -> the experts'
             grouped 4-bit products -> weighted sum back onto the residual

Random weights and inputs; the layer's output is fed back as its next input.

  python examples/rollout_moe.py [--prompts 8 --prompt-tokens 1024 --chunk 512 --steps 64]
"""
import argparse
import os
import sys
import time
from collections import namedtuple

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import fp4_block_quantization_amd as fq

# everything a pass computes, in order
Step = namedtuple("Step", "x qkv q k v attended mixed normed logits weights experts rows offsets place up act down out")


def norm(x):
    y = x.float()
    return (y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6)).bfloat16()


def starts(lens):
    return torch.tensor([0] + lens, device="cuda").cumsum(0).int()


class Layer:
    """Attention with rotary positions, and routed experts, with 4-bit weights."""

    def __init__(self, hidden=2048, heads=32, kv_heads=8, dim=128, experts=64, groups=8, top_groups=4, top_k=8,
                 ffn=512, seed=0):
        self.heads, self.kv_heads, self.dim, self.experts = heads, kv_heads, dim, experts
        self.groups, self.top_groups, self.top_k = groups, top_groups, top_k
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(n, k):
            return (torch.randn((n, k), device="cuda", generator=gen) * k ** -0.5).bfloat16()

        self.qkv = fq.nvfp4_quantize(weight((heads + 2 * kv_heads) * dim, hidden))[:3]
        self.o = fq.nvfp4_quantize(weight(hidden, heads * dim))[:3]
        self.gate = weight(experts, hidden)
        self.bias = 0.05 * torch.randn(experts, device="cuda", generator=gen)  # balances the choice
        self.up = self._experts(weight(experts * 2 * ffn, hidden))
        self.down = self._experts(weight(experts * hidden, ffn))
        self.frequencies, self.amplitude = fq.rotary_frequencies(dim, method="parts", factor=8.0,
                                                                 original_positions=4096)

    def _experts(self, w):
        return [t.view(self.experts, w.shape[0] // self.experts, *t.shape[1:]) for t in fq.nvfp4_quantize(w)[:3]]

    def step(self, x, positions, attend, active=None):
        """x BF16 [tokens, hidden] -> Step; attend(q, k, v) writes the cache and
        gives [tokens, heads, dim]; active: which tokens are no padding."""
        qkv = fq.nvfp4_linear(norm(x), *self.qkv).view(x.shape[0], -1, self.dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        q, k = fq.rotary(q, k, positions, self.frequencies, amplitude=self.amplitude)
        attended = attend(q, k, v)
        mixed = fq.nvfp4_linear(attended.reshape(x.shape[0], -1), *self.o) + x
        normed = norm(mixed)
        logits = torch.nn.functional.linear(normed, self.gate)
        weights, experts = fq.moe_route(logits, self.top_k, bias=self.bias, scoring="sigmoid", groups=self.groups,
                                        top_groups=self.top_groups, active=active)
        rows, offsets, place = fq.moe_dispatch(normed, experts, self.experts)
        up = fq.nvfp4_linear(rows, *self.up, offsets=offsets)
        a, b = up.chunk(2, 1)
        act = torch.nn.functional.silu(a) * b
        down = fq.nvfp4_linear(act, *self.down, offsets=offsets)
        out = fq.moe_combine(down, place, weights, add=mixed)
        return Step(x, qkv, q, k, v, attended, mixed, normed, logits, weights, experts, rows, offsets, place, up, act,
                    down, out)


class Rollout:
    """Sequences with their cache; the batch is padded to `room` of them."""

    def __init__(self, layer, lens, max_tokens, room=None, page=64):
        self.layer, self.page, self.count = layer, page, len(lens)
        room = room or len(lens)
        per = -(-max_tokens // page)
        self.cache = fq.nvfp4_kv_cache(room * per, page, layer.kv_heads, layer.dim)
        self.pages = torch.randperm(room * per, device="cuda").int().view(room, per)
        self.lens = torch.zeros(room, dtype=torch.int32, device="cuda")
        self.active = torch.arange(room, device="cuda") < self.count
        hidden = layer.gate.shape[1]
        self.x = torch.zeros((room, hidden), dtype=torch.bfloat16, device="cuda")

    def slots(self, sequences, at):
        """Cache slots of the sequences' tokens number at."""
        return self.pages[sequences, at // self.page].long() * self.page + at % self.page

    def prefill(self, prompts, chunk):
        """prompts: BF16 [tokens, hidden] of each sequence, put through in chunks.
        Returns the chunks' Steps."""
        steps, done = [], [0] * self.count
        while any(n < len(p) for n, p in zip(done, prompts)):
            new = [min(chunk, len(p) - n) for n, p in zip(done, prompts)]
            x = torch.cat([p[n:n + m] for p, n, m in zip(prompts, done, new)])
            upto = [n + m for n, m in zip(done, new)]
            of = lambda counts: torch.arange(self.count, device="cuda").repeat_interleave(
                torch.tensor(counts, device="cuda"))
            at = torch.cat([torch.arange(n, u, device="cuda") for n, u in zip(done, upto)])
            slots = self.slots(of(new), at)

            def attend(q, k, v):
                fq.nvfp4_kv_append(self.cache, k, v, slots)
                if not any(done):  # the first chunks: their own keys, unrounded
                    return fq.prompt_attention(q, k, v, starts(new))
                back = torch.cat([torch.arange(u, device="cuda") for u in upto])
                k, v = fq.nvfp4_kv_read(self.cache, self.slots(of(upto), back))
                return fq.prompt_attention(q, k, v, starts(new), starts(upto))

            steps.append(self.layer.step(x, at, attend))
            ends = starts(new)[1:].long() - 1
            for i, m in enumerate(new):
                if m:
                    self.x[i] = steps[-1].out[ends[i]]
            done = upto
        self.lens[:self.count] = torch.tensor(done, dtype=torch.int32, device="cuda")
        return steps

    def decode(self):
        """One token of every active sequence: launches only."""
        at = self.lens.long()
        every = torch.arange(self.lens.shape[0], device="cuda")
        slots = torch.where(self.active, self.slots(every, at), -1)
        self.lens += self.active

        def attend(q, k, v):
            fq.nvfp4_kv_append(self.cache, k, v, slots)
            return fq.nvfp4_kv_attention(q, self.cache, self.pages, self.lens)

        step = self.layer.step(self.x, at, attend, self.active)
        self.x.copy_(step.out)
        return step

    def capture(self):
        """decode() as a graph: (graph, the Step its replays write to)."""
        state = [t.clone() for t in (self.x, self.lens)]
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            self.decode()
        torch.cuda.current_stream().wait_stream(stream)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step = self.decode()
        for t, was in zip((self.x, self.lens), state):
            t.copy_(was)
        return graph, step


def main():
    ap = argparse.ArgumentParser()
    for name, value in (("prompts", 8), ("prompt-tokens", 1024), ("chunk", 512), ("steps", 64)):
        ap.add_argument("--" + name, type=int, default=value)
    args = ap.parse_args()
    torch.manual_seed(0)
    layer = Layer()
    lens = [max(1, args.prompt_tokens - 97 * i) for i in range(args.prompts)]
    prompts = [torch.randn((n, 2048), device="cuda").bfloat16() for n in lens]
    Rollout(layer, lens, args.prompt_tokens).prefill(prompts, args.chunk)
    roll = Rollout(layer, lens, args.prompt_tokens + args.steps)
    torch.cuda.synchronize()
    start = time.perf_counter()
    roll.prefill(prompts, args.chunk)
    torch.cuda.synchronize()
    prefill = time.perf_counter() - start
    graph, step = roll.capture()
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(args.steps):
        graph.replay()
    torch.cuda.synchronize()
    seconds = time.perf_counter() - start
    counts = step.offsets.diff()
    print("%d prompts of %d-%d tokens: %.1f ms; decode %.1f us a token of all, %.0f tokens/s; rows of the busiest "
          "expert %d of %d; output rms %.3f" % (
              args.prompts, min(lens), max(lens), prefill * 1e3, seconds / args.steps * 1e6,
              args.prompts * args.steps / seconds, int(counts.max()), int(counts.sum()),
              step.out.float().square().mean().sqrt().item()))


if __name__ == "__main__":
    main()
