"""The layer operators' binding: shapes and types that are refused, gradients,
other streams, two calls at once, and captured graphs."""
import threading

import pytest
import torch

import fp4_block_quantization_amd as fq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fq.rollout_lib()


def bf16(*s):
    return torch.randn(s, device="cuda").bfloat16()


def f32(*s):
    return torch.randn(s, device="cuda")


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def refused(call, good, bad):
    call(**good)
    for kw in bad:
        with pytest.raises(fq.Fp4qError):
            call(**{**good, **kw})


def test_rotary_refuses():
    f, _ = fq.rotary_frequencies(64)
    good = dict(q=bf16(5, 4, 64), k=bf16(5, 2, 64), positions=torch.arange(5, device="cuda"), frequencies=f)
    q = good["q"]
    refused(fq.rotary, good, [
        dict(q=q.half()), dict(q=q.float()), dict(k=good["k"].float()), dict(q=q[0]), dict(k=bf16(4, 2, 64)),
        dict(k=bf16(5, 2, 32)), dict(positions=torch.arange(4, device="cuda")),
        dict(positions=torch.arange(5, dtype=torch.int32, device="cuda")), dict(positions=torch.arange(5)),
        dict(frequencies=f.float()), dict(frequencies=f[:0]), dict(frequencies=f.view(2, 16)), dict(frequencies=f.cpu()),
        dict(frequencies=torch.cat([f, f])), dict(amplitude=float("nan")), dict(q=q.transpose(0, 1)),
        dict(q=q[..., ::2]), dict(q=q[:, ::2], k=None), dict(q=q[:1].expand(5, 4, 64)),
        dict(out=q), dict(out=(q,)), dict(out=(q, None)), dict(out=(q[:4], good["k"])),
        dict(out=(q.float(), good["k"])), dict(k=None, out=(q, good["k"]))])


def test_prompt_refuses():
    good = dict(q=bf16(6, 4, 64), k=bf16(8, 2, 64), v=bf16(8, 2, 64), q_offsets=i32(0, 6), k_offsets=i32(0, 8))
    q, k = good["q"], good["k"]
    refused(fq.prompt_attention, good, [
        dict(q=q.float()), dict(k=k.float()), dict(q=q[None]), dict(k=k[:, :1].expand(8, 2, 64)),
        dict(v=bf16(7, 2, 64)), dict(v=bf16(8, 1, 64)), dict(k=bf16(8, 2, 32)), dict(q=bf16(6, 3, 64)),
        dict(q=bf16(6, 4, 80), k=bf16(8, 2, 80), v=bf16(8, 2, 80)), dict(q_offsets=i32(0, 6).long()),
        dict(q_offsets=i32()), dict(k_offsets=i32(0, 4, 8)), dict(q_offsets=i32(0, 6)[None]), dict(q_offsets=i32(0, 6).cpu()),
        dict(scale=float("inf")), dict(scale=2.0 ** 120), dict(out=bf16(6, 4, 32)), dict(out=q.float()),
        dict(out=bf16(4, 6, 64).transpose(0, 1)), dict(workspace=torch.zeros(4, device="cuda"))])


def test_route_refuses():
    good = dict(logits=f32(6, 16), top_k=3, bias=f32(16), active=torch.ones(6, dtype=torch.bool, device="cuda"))
    refused(fq.moe_route, good, [
        dict(logits=f32(6, 16).half()), dict(logits=f32(16)), dict(logits=f32(16, 6).t()), dict(bias=f32(15)),
        dict(bias=f32(16).bfloat16()), dict(active=torch.ones(5, dtype=torch.bool, device="cuda")),
        dict(active=torch.ones(6, dtype=torch.uint8, device="cuda")), dict(top_k=0), dict(top_k=17), dict(top_k=-1),
        dict(groups=3), dict(groups=4, top_groups=5), dict(groups=8, top_groups=1), dict(scoring="max"),
        dict(scale=float("nan")), dict(out=(f32(6, 3),)), dict(out=(f32(6, 3), i32(0))), dict(bias=f32(16).cpu()),
        dict(out=(f32(6, 3), torch.zeros((6, 3), device="cuda")))])


def test_dispatch_and_combine_refuse():
    e = torch.zeros((6, 2), dtype=torch.int32, device="cuda")
    good = dict(x=bf16(6, 32), experts=e, num_experts=4)
    refused(fq.moe_dispatch, good, [
        dict(x=f32(6, 32)), dict(x=bf16(5, 32)), dict(x=bf16(32, 6).t()), dict(experts=e.long()), dict(experts=e[:, 0]),
        dict(num_experts=0), dict(num_experts=1025), dict(out=(bf16(12, 32),)),
        dict(out=(bf16(11, 32), torch.zeros(5, dtype=torch.int64, device="cuda"), e)),
        dict(out=(bf16(12, 32), i32(0, 0, 0, 0, 0), e)), dict(experts=e.cpu())])
    good = dict(y=bf16(12, 32), place=e, weights=f32(6, 2), add=bf16(6, 32))
    refused(fq.moe_combine, good, [
        dict(y=bf16(12, 32).half()), dict(y=bf16(32)), dict(y=bf16(32, 12).t()), dict(place=e.long()),
        dict(place=e[:, 0]), dict(weights=f32(6, 3)), dict(weights=bf16(6, 2)), dict(add=f32(6, 32)),
        dict(add=bf16(6, 31)), dict(out=bf16(6, 31)), dict(out=f32(6, 32).half()), dict(out_dtype=torch.float16),
        dict(out_dtype=torch.float32, out=bf16(6, 32)), dict(weights=f32(6, 2).cpu())])


def test_gradients_are_refused():
    asks = lambda t: t.clone().requires_grad_()
    f, _ = fq.rotary_frequencies(64)
    pos, off, e = torch.arange(4, device="cuda"), i32(0, 4), torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    q, k, x, w = bf16(4, 4, 64), bf16(4, 2, 64), bf16(4, 32), f32(4, 2)
    calls = [lambda: fq.rotary(asks(q), k, pos, f), lambda: fq.rotary(q, asks(k), pos, f),
             lambda: fq.rotary(q, k, pos, asks(f)), lambda: fq.prompt_attention(asks(q), k, k, off),
             lambda: fq.prompt_attention(q, asks(k), k, off), lambda: fq.prompt_attention(q, k, asks(k) * 2, off),
             lambda: fq.moe_route(asks(x), 2), lambda: fq.moe_route(x, 2, bias=asks(f32(32))),
             lambda: fq.moe_dispatch(asks(x), e, 3), lambda: fq.moe_combine(asks(x), e, w),
             lambda: fq.moe_combine(x, e, asks(w)), lambda: fq.moe_combine(x, e, w, add=asks(x))]
    for call in calls:
        with pytest.raises(fq.Fp4qError, match="gradient"):
            call()
        with torch.no_grad():
            call()
        with torch.inference_mode():
            call()


def work(seed):
    """Inputs of every operator, and one pass over them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    f, a = fq.rotary_frequencies(128, method="parts", factor=4.0, original_positions=4096)
    t = dict(q=rnd(300, 8, 128).bfloat16(), k=rnd(300, 2, 128).bfloat16(), v=rnd(300, 2, 128).bfloat16(),
             pos=torch.arange(300, device="cuda") + 5000, off=i32(0, 100, 101, 300), ck=rnd(6000, 2, 128).bfloat16(),
             cv=rnd(6000, 2, 128).bfloat16(), coff=i32(0, 2000, 2500, 6000), one=i32(0, 1, 2, 3), logits=rnd(700, 64), bias=0.1 * rnd(64),
             x=rnd(700, 96).bfloat16(), y=rnd(700 * 8, 96).bfloat16())

    def run():
        q, k = fq.rotary(t["q"], t["k"], t["pos"], f, amplitude=a)
        o = fq.prompt_attention(q, k, t["v"], t["off"])
        # contexts in parts, with a workspace
        c = fq.prompt_attention(q[:3], t["ck"], t["cv"], t["one"], t["coff"])
        w, e = fq.moe_route(t["logits"], 8, bias=t["bias"], scoring="sigmoid", groups=8, top_groups=4)
        rows, offsets, place = fq.moe_dispatch(t["x"], e, 64)
        return q, k, o, c, w, e, rows, offsets, place, fq.moe_combine(t["y"], place, w, add=t["x"])

    return t, run


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def test_same_bits_from_call_to_call_and_on_other_streams():
    t, run = work(1)
    want = [x.clone() for x in run()]
    assert same(run(), want)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):  # several at once
        for s in streams:
            with torch.cuda.stream(s):
                got.append(run())
    torch.cuda.synchronize()
    for g in got:
        assert same(g, want)


def test_graphs_replay():
    t, run = work(2)
    fresh = {k: v.clone() for k, v in work(3)[0].items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    with torch.cuda.graph(second):  # another graph of the same calls, with workspaces of its own
        out2 = run()
    first = {k: v.clone() for k, v in t.items()}
    for i in range(6):
        for name, v in (fresh if i % 2 else first).items():
            t[name].copy_(v)
        want = [x.clone() for x in run()]  # eager work between the replays
        graph.replay()
        second.replay()
        if i % 3 == 0:
            torch.cuda.synchronize()
        assert same(out, want) and same(out2, want), i


def test_lengths_that_change_between_replays():
    # the offsets are read on the device: a graph of one capacity serves any lengths within it
    q, k, v = bf16(200, 4, 64), bf16(200, 2, 64), bf16(200, 2, 64)
    off = i32(0, 200, 200, 200)
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fq.prompt_attention(q, k, v, off, out=out)
    for lens in ((0, 50, 120, 130), (0, 0, 0, 7), (10, 110, 110, 200), (0, 200, 200, 200)):
        off.copy_(i32(*lens))
        out.fill_(5.0)
        graph.replay()
        want = fq.prompt_attention(q, k, v, off, out=torch.full_like(q, 5.0))
        assert torch.equal(out, want)
        assert (out[:lens[0]] == 5).all() and (out[lens[3]:] == 5).all()


def test_inactive_padding_in_a_graph():
    # a batch padded to the graph's size: routing, rows and sums of the padding are empty
    x, logits = bf16(32, 64), f32(32, 16)
    active = torch.ones(32, dtype=torch.bool, device="cuda")
    y = bf16(32 * 4, 64)
    rows = torch.zeros((128, 64), dtype=torch.bfloat16, device="cuda")
    off, place = torch.empty(17, dtype=torch.int64, device="cuda"), torch.empty((32, 4), dtype=torch.int32, device="cuda")

    def step():
        w, e = fq.moe_route(logits, 4, active=active)
        fq.moe_dispatch(x, e, 16, out=(rows, off, place))
        return w, fq.moe_combine(y, place, w)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w, out = step()
    for n in (32, 5, 0, 31):
        active.copy_(torch.arange(32, device="cuda") < n)
        rows.fill_(9.0)
        graph.replay()
        assert int(off[-1]) == 4 * n and (place[n:] == -1).all() and (w[n:] == 0).all()
        assert (out[n:] == 0).all() and (rows[4 * n:] == 9).all()
        assert torch.equal(rows[place[:n].long()], x[:n, None].expand(n, 4, 64))


def test_small_outputs_of_a_call_share_an_allocation_and_nothing_else():
    f, _ = fq.rotary_frequencies(64)

    def calls(tokens):
        x = torch.randn((tokens, 6, 64), device="cuda").bfloat16()
        p = torch.arange(tokens, device="cuda")
        yield fq.rotary(x[:, :4], x[:, 4:], p, f)
        yield fq.prompt_attention(x[:, :4], x[:, 4:5], x[:, 5:], torch.tensor([0, tokens], device="cuda").int(),
                                  lse=True)
        w, e = fq.moe_route(torch.randn((tokens, 9), device="cuda"), 3)
        yield w, e
        yield fq.moe_dispatch(x.view(tokens, 384), e, 9)[1:]

    for tokens in (0, 1, 7, 300):
        for outs in calls(tokens):
            assert len({t.untyped_storage().data_ptr() for t in outs}) == 1
            ends = [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in outs if t.numel()]
            assert all(a % 16 == 0 for a, _ in ends)
            assert all(b <= c or d <= a for i, (a, b) in enumerate(ends) for c, d in ends[i + 1:])
            assert all(t.is_contiguous() and not t.requires_grad and not t._is_view() for t in outs)
            kept = [t.clone() for t in outs]
            outs[0].fill_(3)
            assert torch.equal(outs[1], kept[1])
            outs[1].zero_()
            assert (outs[0] == 3).all()
    # larger ones do not keep each other's memory
    q, k = next(calls(20000))
    assert q.untyped_storage().data_ptr() != k.untyped_storage().data_ptr()
    assert q.storage_offset() == k.storage_offset() == 0


def test_calls_in_inference_mode_and_from_threads():
    def chain(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x = torch.randn((130, 6, 64), generator=g, device="cuda").bfloat16()
        f, a = fq.rotary_frequencies(64)
        q, k = fq.rotary(x[:, :4], x[:, 4:5], torch.arange(130, device="cuda"), f, amplitude=a)
        off = torch.tensor([0, 30, 130], dtype=torch.int32, device="cuda")
        o, lse = fq.prompt_attention(q, k, x[:, 5:], off, lse=True)
        w, e = fq.moe_route(o.view(130, 256).float(), 4)
        rows, offsets, place = fq.moe_dispatch(o.view(130, 256), e, 256)
        return q, k, o, lse, w, e, rows, offsets, place, fq.moe_combine(rows, place, w, add=o.view(130, 256))

    want = [chain(i) for i in range(4)]
    with torch.inference_mode():
        got = chain(0)
        assert all(t.is_inference() for t in got)
        assert all(torch.equal(a, b) for a, b in zip(want[0], got))
        got[0].add_(1)
    results = [None] * 4

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                results[i] = chain(i)
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(4):
        assert all(torch.equal(a, b) for a, b in zip(want[i], results[i]))
