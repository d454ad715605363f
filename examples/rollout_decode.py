"""Rollout decoding with the 4-bit operators: one transformer layer generates
several samples for each of a few prompts.

  weights    quantized once: attention to NVFP4, the experts' to MXFP4
  prefill    the prompts' keys and values go into the cache, once per prompt
  decode     fused QKV product -> cache write -> attention over the prompt
             (shared by its samples) and the sample's own tokens -> output
             product -> the experts' grouped products; one captured HIP graph
             that is replayed for every token
  hand-over  a sample's keys and values read back in BF16

Random weights and inputs; the layer's output is fed back as its next input,
in place of an embedding.

  python examples/rollout_decode.py [--prompts 4 --samples 16 --prompt-tokens 1024 --steps 64]
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

# everything a step computes, in order: inputs and outputs of the five operators' calls
Step = namedtuple("Step", "x qkv attended mixed routed up act down out")


def norm(x):
    y = x.float()
    return (y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6)).bfloat16()


class Layer:
    """Attention and routed experts with 4-bit weights."""

    def __init__(self, hidden=2048, heads=32, kv_heads=8, dim=128, experts=8, ffn=1024, seed=0):
        self.heads, self.kv_heads, self.dim, self.experts = heads, kv_heads, dim, experts
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(n, k):
            w = torch.randn((n, k), device="cuda", generator=gen)
            return (w * k ** -0.5).bfloat16()

        # codes, block scales and row scales of W [n, k]
        self.qkv = fq.nvfp4_quantize(weight((heads + 2 * kv_heads) * dim, hidden))[:3]
        self.o = fq.nvfp4_quantize(weight(hidden, heads * dim))[:3]
        # codes and scales of every expert's matrix, [experts, n, ..]
        self.up = self._experts(weight(experts * ffn, hidden))
        self.down = self._experts(weight(experts * hidden, ffn))

    def _experts(self, w):
        codes, scales = fq.mxfp4_resq_quantize(w)[:2]
        return [t.view(self.experts, w.shape[0] // self.experts, -1) for t in (codes, scales)]

    def step(self, x, cache, slots, pages, lens, order, offsets, prefix=None):
        """x BF16 [batch, tokens, hidden] -> Step.  slots: where the tokens go;
        pages and lens (with the new tokens): what a sequence reads; order:
        the token of each routed row, grouped by expert at offsets."""
        batch, tokens, hidden = x.shape
        qkv = fq.nvfp4_linear(norm(x).view(-1, hidden), *self.qkv)
        rows = qkv.view(batch * tokens, -1, self.dim)
        q, k, v = rows.split([self.heads, self.kv_heads, self.kv_heads], 1)
        fq.nvfp4_kv_append(cache, k, v, slots)
        q = q.view(batch, tokens, self.heads, self.dim)  # a strided slice, taken as it lies
        attended = fq.nvfp4_kv_attention(q, cache, pages, lens, prefix=prefix)
        mixed = fq.nvfp4_linear(attended.view(batch * tokens, -1), *self.o)
        mixed = mixed + x.view(-1, hidden)
        routed = norm(mixed)[order]
        up = fq.mxfp4_linear(routed, *self.up, offsets=offsets)
        act = torch.nn.functional.silu(up)
        down = fq.mxfp4_linear(act, *self.down, offsets=offsets)
        out = mixed.index_copy(0, order, mixed[order] + down)
        return Step(x, qkv, attended, mixed, routed, up, act, down, out.view(x.shape))


class Rollout:
    """A cache with the prompts in it, and the samples' state."""

    def __init__(self, layer, prompts, samples, steps, page=64):
        """prompts: BF16 [prompts, tokens, hidden]."""
        self.layer, self.page = layer, page
        n, length, hidden = prompts.shape
        batch = n * samples
        own, shared = -(-steps // page), -(-length // page)
        self.cache = fq.nvfp4_kv_cache(n * shared + batch * own, page, layer.kv_heads, layer.dim)
        ids = torch.arange(n * shared + batch * own, dtype=torch.int32, device="cuda")
        self.prompt_pages = ids[:n * shared].view(n, shared)
        self.pages = ids[n * shared:].view(batch, own)
        lens = torch.full((n,), length, dtype=torch.int32, device="cuda")
        place = torch.arange(length, device="cuda")
        slots = self.prompt_pages.long()[:, place // page] * page + place % page
        self.prefill = layer.step(prompts, self.cache, slots.view(-1), self.prompt_pages, lens,
                                  *self._route(n * length))
        members = torch.arange(0, batch + 1, samples, dtype=torch.int32, device="cuda")
        self.prefix = (self.prompt_pages, lens, members)
        self.route = self._route(batch)
        # each sample starts from its prompt's last output, told apart by a little noise
        first = self.prefill.out[:, -1:].repeat_interleave(samples, 0)
        self.start = (first + 0.1 * torch.randn(first.shape, device="cuda")).bfloat16()
        self.x = torch.empty_like(self.start)
        self.lens = torch.empty(batch, dtype=torch.int32, device="cuda")
        self.reset()

    def _route(self, rows):
        # a fixed, uneven choice of experts
        expert = (torch.arange(rows) ** 2) % self.layer.experts
        counts = torch.bincount(expert, minlength=self.layer.experts)
        offsets = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
        return expert.argsort(stable=True).cuda(), offsets.cuda()

    def reset(self):
        self.x.copy_(self.start)
        self.lens.zero_()

    def slots(self, at):
        """The cache slots of the samples' tokens number at [batch]."""
        page = self.pages.gather(1, (at // self.page).long()[:, None])[:, 0]
        return page.long() * self.page + at % self.page

    def decode(self):
        """One token of every sample: launches only, nothing waits for the host."""
        slots = self.slots(self.lens)
        self.lens += 1
        step = self.layer.step(self.x, self.cache, slots, self.pages, self.lens, *self.route,
                               prefix=self.prefix)
        self.x.copy_(step.out)
        return step

    def capture(self):
        """decode() as a graph: (graph, the Step its replays write to)."""
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            self.decode()
        torch.cuda.current_stream().wait_stream(stream)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step = self.decode()
        self.reset()
        return graph, step


def main():
    ap = argparse.ArgumentParser()
    for name, value in (("prompts", 4), ("samples", 16), ("prompt-tokens", 1024), ("steps", 64)):
        ap.add_argument("--" + name, type=int, default=value)
    args = ap.parse_args()
    torch.manual_seed(0)
    layer = Layer()
    prompts = torch.randn((args.prompts, args.prompt_tokens, 2048), device="cuda").bfloat16()
    roll = Rollout(layer, prompts, args.samples, args.steps)
    graph, step = roll.capture()
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(args.steps):
        graph.replay()
    torch.cuda.synchronize()
    seconds = time.perf_counter() - start
    k, v = fq.nvfp4_kv_read(roll.cache, roll.slots(torch.zeros_like(roll.lens)))
    bits = 8 * sum(t.numel() * t.element_size() for t in roll.cache)
    values = 2 * 2 * roll.cache.k_codes.numel()
    print("%d samples x %d tokens on %d prompts of %d: %.1f us a token of all samples, %.0f "
          "tokens/s; cache %.2f bits a value; first tokens' keys and values %s; output rms %.3f" % (
              args.prompts * args.samples, args.steps, args.prompts, args.prompt_tokens,
              seconds / args.steps * 1e6, args.prompts * args.samples * args.steps / seconds,
              bits / values, tuple(k.shape), step.out.float().square().mean().sqrt().item()))


if __name__ == "__main__":
    main()
