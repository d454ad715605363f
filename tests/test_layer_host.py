"""The calls of include/fp4q/layer.h are exported, and reject bad arguments on
the host before any HIP call (no GPU needed; nothing here launches a kernel)."""
import ctypes
import math
import os
import re

import pytest
import torch

import fp4_block_quantization_amd as fq
from fp4_block_quantization_amd import layer

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SUCCESS, NULL, SHAPE, MISALIGNED, LAUNCH, INVALID = 0, 1, 2, 3, 4, 5
P = ctypes.c_void_p
A16, B16, A8, A4, A2, ODD = P(0x10000), P(0x20000), P(0x10008), P(0x10004), P(0x10002), P(0x10001)


def lib():
    return layer.declare(fq.rollout_lib())


def test_library_exports_every_declared_call():
    src = open(os.path.join(ROOT, "include", "fp4q", "layer.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"FP4Q_API\s+\w+\s+(\w+)\s*\(", src)))
    assert names == ["moe_combine", "moe_dispatch", "moe_dispatch_workspace_bytes", "moe_route",
                     "prompt_attention", "prompt_attention_workspace_bytes", "rotary_embed"]
    for n in names:
        assert hasattr(lib(), n), n


def call(name, defaults):
    def f(**kw):
        assert set(kw) <= set(defaults), kw
        return getattr(lib(), name)(*{**defaults, **kw}.values())
    return f


rotary = call("rotary_embed", dict(
    q=A16, q_stride=512, q_heads=4, k=A16, k_stride=256, k_heads=2, tokens=3, dim=128, dims=128,
    positions=A8, frequencies=A8, amplitude=1.0, interleaved=0, inverse=0, fp32=0, q_out=B16,
    q_out_stride=512, k_out=B16, k_out_stride=256, stream=None))
prompt = call("prompt_attention", dict(
    q=A16, q_stride=512, q_tokens=5, q_heads=4, k=A16, k_stride=256, v=A16, v_stride=256,
    k_tokens=5, kv_heads=2, dim=128, q_off=A4, k_off=A4, batch=2, scale=0.1, out=B16, lse=None,
    ws=A16, ws_bytes=1 << 40, stream=None))
route = call("moe_route", dict(
    logits=A4, fp32=1, tokens=3, experts=64, top_k=4, bias=None, scoring=0, groups=1, top_groups=1,
    renormalize=1, scale=1.0, active=None, weights=A4, chosen=A4, stream=None))
dispatch = call("moe_dispatch", dict(
    x=A16, tokens=3, hidden=64, chosen=A4, top_k=2, experts=8, rows=B16, offsets=A8, place=A4,
    ws=A16, ws_bytes=1 << 40, stream=None))
combine = call("moe_combine", dict(
    y=A16, y_fp32=0, y_rows=6, place=A4, weights=A4, add=None, tokens=3, top_k=2, n=64, out_fp32=0,
    out=B16, stream=None))


def test_rotary_rejects():
    for kw in (dict(tokens=-1), dict(q_heads=0), dict(k_heads=-1), dict(dim=0), dict(dims=0),
               dict(dims=127), dict(dims=130), dict(q_stride=511), dict(k_stride=255),
               dict(q_out_stride=511), dict(k_out_stride=0), dict(q_heads=70000, q_stride=1 << 40),
               dict(tokens=1 << 31), dict(tokens=1 << 30, q_stride=1 << 20)):
        assert rotary(**kw) == SHAPE, kw
    for name in ("interleaved", "inverse", "fp32"):
        assert rotary(**{name: 2}) == INVALID
    for a in (math.nan, math.inf):
        assert rotary(amplitude=a) == INVALID
    for name in ("q", "k", "q_out", "k_out", "positions", "frequencies"):
        assert rotary(**{name: None}) == NULL, name
    for name in ("q", "k", "q_out", "k_out"):
        assert rotary(**{name: ODD}) == MISALIGNED
        assert rotary(**{name: A2}, fp32=1) == MISALIGNED
    assert rotary(positions=A4) == MISALIGNED
    assert rotary(frequencies=A4) == MISALIGNED
    # in place, but from rows that lie otherwise
    assert rotary(q_out=A16, q_out_stride=640) == INVALID
    assert rotary(k_out=A16, k_out_stride=640) == INVALID
    assert rotary(tokens=0, q=None, k=None, q_out=None, k_out=None, positions=None,
                  frequencies=None) == SUCCESS


def test_prompt_rejects():
    for kw in (dict(dim=80), dict(q_heads=3), dict(q_heads=0), dict(kv_heads=0), dict(batch=-1),
               dict(batch=70000), dict(q_tokens=-1), dict(k_tokens=-1), dict(q_tokens=1 << 31),
               dict(q_stride=504), dict(q_stride=516), dict(k_stride=248), dict(v_stride=260),
               dict(k_stride=(1 << 24) + 8), dict(q_tokens=1 << 30, q_heads=4, kv_heads=1),
               dict(q_tokens=1 << 30, q_heads=64, kv_heads=64, q_stride=8192, k_stride=8192,
                    v_stride=8192)):
        assert prompt(**kw) == SHAPE, kw
    for s in (math.nan, math.inf, -math.inf, 2.0 ** 101):
        assert prompt(scale=s) == INVALID
    for name in ("q", "k", "v", "q_off", "k_off", "out"):
        assert prompt(**{name: None}) == NULL, name
    for name in ("q", "k", "v", "out"):
        assert prompt(**{name: A8}) == MISALIGNED, name
    assert prompt(q_off=A2) == MISALIGNED
    assert prompt(k_off=A2) == MISALIGNED
    assert prompt(lse=A2) == MISALIGNED
    nothing = dict(q=None, k=None, v=None, q_off=None, k_off=None, out=None, ws=None)
    assert prompt(batch=0, **nothing) == SUCCESS
    assert prompt(q_tokens=0, **nothing) == SUCCESS
    need = lib().prompt_attention_workspace_bytes
    assert need(5, 4, 5, 2, 80, 2) == 0  # sizes the call refuses


def test_route_rejects():
    for kw in (dict(tokens=-1), dict(experts=0), dict(experts=1025), dict(top_k=0), dict(top_k=65),
               dict(experts=3, top_k=4), dict(groups=0), dict(groups=7), dict(groups=65, experts=130),
               dict(groups=8, top_groups=9), dict(groups=8, top_groups=0),
               dict(groups=32, top_groups=1, top_k=4)):
        assert route(**kw) == SHAPE, kw
    for name in ("fp32", "scoring", "renormalize"):
        assert route(**{name: 2}) == INVALID, name
    assert route(scale=math.nan) == INVALID
    for name in ("logits", "weights", "chosen"):
        assert route(**{name: None}) == NULL, name
        assert route(**{name: A2}) == MISALIGNED, name
    assert route(bias=A2) == MISALIGNED
    assert route(logits=ODD, fp32=0) == MISALIGNED
    assert route(tokens=0, logits=None, weights=None, chosen=None) == SUCCESS


def test_dispatch_rejects():
    for kw in (dict(tokens=-1), dict(hidden=0), dict(top_k=0), dict(top_k=65), dict(experts=0),
               dict(experts=1025), dict(tokens=1 << 30), dict(tokens=1 << 20, hidden=1 << 20)):
        assert dispatch(**kw) == SHAPE, kw
    for name in ("x", "chosen", "rows", "offsets", "place"):
        assert dispatch(**{name: None}) == NULL, name
    assert dispatch(x=ODD) == MISALIGNED
    assert dispatch(rows=ODD) == MISALIGNED
    assert dispatch(offsets=A4) == MISALIGNED
    assert dispatch(chosen=A2) == MISALIGNED
    assert dispatch(place=A2) == MISALIGNED
    assert dispatch(ws=A8) == MISALIGNED
    need = lib().moe_dispatch_workspace_bytes(1 << 20, 8, 64)
    assert need > 0
    many = dict(tokens=1 << 20, top_k=8, experts=64)
    assert dispatch(**many, ws=None) == NULL
    assert dispatch(**many, ws_bytes=need - 1) == INVALID
    assert lib().moe_dispatch_workspace_bytes(8, 65, 64) == 0  # sizes the call refuses


def test_combine_rejects():
    for kw in (dict(tokens=-1), dict(y_rows=-1), dict(y_rows=1 << 31), dict(top_k=0),
               dict(top_k=65), dict(n=0), dict(tokens=1 << 30, n=1 << 20)):
        assert combine(**kw) == SHAPE, kw
    for name in ("y_fp32", "out_fp32"):
        assert combine(**{name: 2}) == INVALID, name
    for name in ("y", "place", "weights", "out"):
        assert combine(**{name: None}) == NULL, name
    for name in ("y", "add", "out"):
        assert combine(**{name: ODD}) == MISALIGNED, name
    assert combine(y=A2, y_fp32=1) == MISALIGNED
    assert combine(out=A2, out_fp32=1) == MISALIGNED
    assert combine(add=B16, out_fp32=1) == INVALID  # BF16 read where FP32 is written
    assert combine(tokens=0, y=None, place=None, weights=None, out=None) == SUCCESS


def test_binding_refuses_tensors_off_the_gpu():
    b, i = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64)
    f, a = fq.rotary_frequencies(64, device="cpu")
    off = torch.zeros(2, dtype=torch.int32)
    e = torch.zeros((4, 2), dtype=torch.int32)
    for c in (lambda: fq.rotary(b, b, i, f), lambda: fq.prompt_attention(b, b, b, off),
              lambda: fq.moe_route(b[:, 0], 2), lambda: fq.moe_dispatch(b[:, 0], e, 3),
              lambda: fq.moe_combine(b[:, 0], e, e.float())):
        with pytest.raises(fq.Fp4qError):
            c()
    with pytest.raises(fq.Fp4qError):
        fq.moe_route(b[:, 0], 2, scoring="max")


def test_frequencies():
    f, a = fq.rotary_frequencies(8, base=100.0, device="cpu")
    assert a == 1.0 and f.dtype is torch.float64
    assert f.tolist() == [100.0 ** (-i / 4) for i in range(4)]
    g, a = fq.rotary_frequencies(8, base=100.0, method="positions", factor=4.0, device="cpu")
    assert a == 1.0 and torch.equal(g, f / 4)
    g, a = fq.rotary_frequencies(8, base=100.0, method="base", factor=4.0, device="cpu")
    assert g[0] == 1.0 and math.isclose(g[3], f[3] / 4, rel_tol=1e-12)
    # 1, 0.316, 0.1, 0.0316 radians a position: 16, 5, 1.6 and 0.5 turns within 100
    g, a = fq.rotary_frequencies(8, base=100.0, method="parts", factor=4.0, original_positions=100,
                                 slow=1.0, fast=10.0, device="cpu")
    assert math.isclose(a, 0.1 * math.log(4.0) + 1)
    assert g[0] == f[0] and math.isclose(g[3], f[3] / 4)
    for i in (1, 2):
        share = (100 * f[i] / (2 * math.pi) - 1) / 9
        assert math.isclose(g[i], f[i] * share + f[i] / 4 * (1 - share), rel_tol=1e-12)
    assert fq.rotary_frequencies(8, method="parts", factor=4.0, original_positions=100,
                                 amplitude=1.0, device="cpu")[1] == 1.0
    for kw in (dict(dims=7), dict(dims=0), dict(dims=8, method="other"), dict(dims=8, factor=0.0),
               dict(dims=8, base=-1.0), dict(dims=8, method="parts"), dict(dims=2, method="base"),
               dict(dims=8, method="parts", original_positions=10, slow=2.0, fast=1.0)):
        with pytest.raises(fq.Fp4qError):
            fq.rotary_frequencies(device="cpu", **kw)
