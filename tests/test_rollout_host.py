"""The rollout library loads, exports every call include/fp4q/rollout.h
declares, and rejects bad arguments on the host before any HIP call (no GPU
needed; nothing here launches a kernel)."""
import ctypes
import os
import re

import pytest
import torch

import fp4_block_quantization_amd as fq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SUCCESS, NULL, SHAPE, MISALIGNED, LAUNCH, INVALID = 0, 1, 2, 3, 4, 5
P = ctypes.c_void_p
A16, A8, A4, ODD = P(0x10000), P(0x10008), P(0x10004), P(0x10001)


def test_library_exports_every_declared_call():
    src = open(os.path.join(ROOT, "include", "fp4q", "rollout.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"FP4Q_API\s+\w+\s+(\w+)\s*\(", src)))
    assert names == ["mxfp4_linear", "mxfp4_linear_workspace_bytes", "nvfp4_kv_append",
                     "nvfp4_kv_attention", "nvfp4_kv_attention_workspace_bytes",
                     "nvfp4_kv_read", "nvfp4_linear", "nvfp4_linear_workspace_bytes"]
    for n in names:
        assert hasattr(fq.rollout_lib(), n), n


def linear(mx=False, x=A16, rows=4, codes=A16, scales=A16, rs=A16, n=32, k=64, offs=None, groups=0,
           f32=0, out=A16, ws=A16, ws_bytes=1 << 40):
    L = fq.rollout_lib()
    if mx:
        return L.mxfp4_linear(x, rows, codes, scales, n, k, offs, groups, f32, out, ws, ws_bytes,
                              None)
    return L.nvfp4_linear(x, rows, codes, scales, rs, n, k, offs, groups, f32, out, ws, ws_bytes,
                          None)


@pytest.mark.parametrize("mx", [False, True])
def test_linear_rejects(mx):
    f = lambda **kw: linear(mx, **kw)
    assert f(k=48 if mx else 40) == SHAPE
    assert f(k=0) == SHAPE
    assert f(n=0) == SHAPE
    assert f(rows=-1) == SHAPE
    assert f(groups=-1) == SHAPE
    assert f(groups=70000, offs=A8) == SHAPE
    assert f(offs=A8) == SHAPE        # offsets without groups
    assert f(groups=2) == NULL        # groups without offsets
    assert f(n=1 << 30, k=1 << 20) == SHAPE
    assert f(f32=2) == INVALID
    assert f(x=None) == NULL
    assert f(codes=None) == NULL
    assert f(scales=None) == NULL
    assert f(out=None) == NULL
    if not mx:
        assert f(rs=None) == NULL
        assert f(rs=P(0x10002)) == MISALIGNED
    assert f(x=A8) == MISALIGNED
    assert f(codes=A8 if mx else A4) == MISALIGNED
    assert f(out=ODD) == MISALIGNED
    assert f(out=P(0x10002), f32=1) == MISALIGNED
    assert f(offs=A4, groups=1) == MISALIGNED
    assert f(ws=A8) == MISALIGNED
    assert f(rows=0, x=None, codes=None, scales=None, rs=None, out=None, ws=None) == SUCCESS
    L = fq.rollout_lib()
    need = L.mxfp4_linear_workspace_bytes if mx else L.nvfp4_linear_workspace_bytes
    assert need(4, 32, 40, 0) == 0    # sizes the call refuses
    big = need(4096, 64, 8192, 0)
    if big > 0:
        assert f(rows=4096, n=64, k=8192, ws_bytes=big - 1) == INVALID
        assert f(rows=4096, n=64, k=8192, ws=None) == NULL


CACHE = dict(kc=A16, ks=A16, kt=A16, vc=A16, vs=A16, vt=A16, pages=4, page=16, heads=2, dim=64)


def cache_args(kw):
    return [kw.pop(n, CACHE[n]) for n in CACHE]


def append(**kw):
    c = cache_args(kw)
    return fq.rollout_lib().nvfp4_kv_append(
        *c, kw.get("k", A16), kw.get("k_stride", 128), kw.get("v", A16), kw.get("v_stride", 128),
        kw.get("tokens", 3), kw.get("slots", A8), kw.get("fos", 1), None)


def read(**kw):
    c = cache_args(kw)
    return fq.rollout_lib().nvfp4_kv_read(*c, kw.get("slots", A8), kw.get("tokens", 3),
                                          kw.get("k", A16), kw.get("v", A16), None)


def attend(**kw):
    c = cache_args(kw)
    return fq.rollout_lib().nvfp4_kv_attention(
        *c, kw.get("q", A16), kw.get("q_stride", 256), kw.get("batch", 2), kw.get("t", 1),
        kw.get("q_heads", 4), kw.get("table", A4), kw.get("max_pages", 3), kw.get("lens", A4),
        kw.get("ptable", None), kw.get("ppages", 0), kw.get("plens", None),
        kw.get("offs", None), kw.get("groups", 0), kw.get("scale", 0.1), kw.get("out", A16),
        kw.get("lse", None), kw.get("ws", A16), kw.get("ws_bytes", 1 << 40), None)


@pytest.mark.parametrize("f", [append, read, attend])
def test_cache_rejects(f):
    assert f(pages=0) == SHAPE
    assert f(page=24) == SHAPE
    assert f(page=0) == SHAPE
    assert f(heads=0) == SHAPE
    assert f(dim=72) == SHAPE
    assert f(dim=528) == SHAPE
    assert f(pages=1 << 28, page=16) == SHAPE  # 2^32 slots
    for name in ("kc", "ks", "kt", "vc", "vs", "vt"):
        assert f(**{name: None}) == NULL, name
    assert f(kc=A8) == MISALIGNED
    assert f(vc=A8) == MISALIGNED
    assert f(vs=P(0x10002)) == MISALIGNED
    assert f(kt=A8) == MISALIGNED


def test_append_and_read_reject():
    assert append(tokens=-1) == SHAPE
    assert append(k_stride=120) == SHAPE
    assert append(v_stride=132) == SHAPE
    assert append(fos=2) == INVALID
    assert append(k=None) == NULL
    assert append(slots=None) == NULL
    assert append(k=A8) == MISALIGNED
    assert append(slots=A4) == MISALIGNED
    assert append(tokens=0, k=None, v=None, slots=None) == SUCCESS
    assert read(tokens=-1) == SHAPE
    assert read(k=None) == NULL
    assert read(v=A8) == MISALIGNED
    assert read(slots=A4) == MISALIGNED
    assert read(tokens=0, k=None, v=None, slots=None) == SUCCESS


def test_attention_rejects():
    assert attend(dim=80, q_stride=320) == SHAPE
    assert attend(q_heads=3) == SHAPE
    assert attend(q_heads=0) == SHAPE
    assert attend(q_stride=248) == SHAPE
    assert attend(q_stride=260) == SHAPE
    assert attend(batch=-1) == SHAPE
    assert attend(t=-1) == SHAPE
    assert attend(batch=70000) == SHAPE
    assert attend(max_pages=-1) == SHAPE
    assert attend(max_pages=1 << 28) == SHAPE
    assert attend(ppages=1) == SHAPE          # a prefix without groups
    assert attend(plens=A4) == SHAPE
    assert attend(scale=float("nan")) == INVALID
    assert attend(scale=float("inf")) == INVALID
    assert attend(q=None) == NULL
    assert attend(lens=None) == NULL
    assert attend(table=None) == NULL
    assert attend(out=None) == NULL
    prefix = dict(groups=1, ppages=2, ptable=A4, plens=A4, offs=A4)
    for name in ("ptable", "plens", "offs"):
        assert attend(**{**prefix, name: None}) == NULL, name
    assert attend(q=A8) == MISALIGNED
    assert attend(out=A8) == MISALIGNED
    assert attend(lens=P(0x10002)) == MISALIGNED
    assert attend(table=ODD) == MISALIGNED
    assert attend(lse=ODD) == MISALIGNED
    assert attend(batch=0, q=None, out=None, lens=None, table=None) == SUCCESS
    assert attend(t=0, q=None, out=None, lens=None, table=None) == SUCCESS
    need = fq.rollout_lib().nvfp4_kv_attention_workspace_bytes
    assert need(16, 2, 80, 2, 1, 4, 3, 0, 0) == 0  # sizes the call refuses
    # a workspace that is missing or too short, where the sizes ask for one
    if need(16, 2, 64, 2, 1, 4, 3, 2, 1) > 0:
        assert attend(**prefix, ws=None) == NULL
        assert attend(**prefix, ws_bytes=0) == INVALID


def test_binding_refuses():
    b = torch.zeros(4, 64, dtype=torch.bfloat16)
    c = fq.nvfp4_kv_cache(2, 16, 2, 64, device="cpu")
    with pytest.raises(fq.Fp4qError):
        fq.nvfp4_linear(b, torch.zeros(8, 32, dtype=torch.uint8),
                        torch.zeros(8, 4, dtype=torch.uint8), torch.zeros(8))
    with pytest.raises(fq.Fp4qError):
        fq.nvfp4_kv_append(c, b.view(2, 2, 64), b.view(2, 2, 64), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(fq.Fp4qError):
        fq.nvfp4_kv_read(c, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(fq.Fp4qError):
        fq.nvfp4_kv_attention(b.view(1, 4, 64), c, torch.zeros(1, 1, dtype=torch.int32),
                              torch.zeros(1, dtype=torch.int32))


def test_cache_shapes():
    c = fq.nvfp4_kv_cache(3, 32, 2, 80, device="cpu")
    assert c.k_codes.shape == c.v_codes.shape == (3, 2, 32, 40)
    assert c.k_scales.shape == (3, 2, 32, 5) and c.v_scales.shape == (3, 2, 5, 32)
    assert c.k_token_scales.shape == c.v_token_scales.shape == (3, 2, 32)


def test_extents_past_the_offsets_are_rejected():
    for f in (append, read, attend):
        assert f(heads=65536, q_stride=1 << 25, q_heads=65536) == SHAPE
    wide = dict(q_stride=256)
    assert attend(pages=1, page=(1 << 27) + 16, **wide) == SHAPE
    assert attend(max_pages=(1 << 26) + 1, **wide) == SHAPE      # more than 2^30 tokens of 16
    assert attend(groups=1, ppages=(1 << 26) + 1, ptable=A4, plens=A4, offs=A4, **wide) == SHAPE
    for mx in (False, True):
        assert linear(mx=mx, rows=1, n=1, k=(1 << 26) + 32) == SHAPE
