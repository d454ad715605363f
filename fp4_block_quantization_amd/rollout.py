"""Operators of a 4-bit rollout engine -- Python binding of
libfp4q_rollout.so (C ABI in include/fp4q/rollout.h).

Argument marshalling only, in the manner of the package's other calls: GPU
tensors in, outputs allocated on the inputs' device or passed in, launches
on torch's current stream, no CPU fallback.

  nvfp4_linear(x, codes, block_scales, row_scales, offsets=None) -> [R, N]
  mxfp4_linear(x, codes, scales, offsets=None) -> [R, N]
  nvfp4_kv_cache(num_pages, page_size, kv_heads, head_dim) -> NvFp4KvCache
  nvfp4_kv_append(cache, k, v, slots, four_over_six=True)
  nvfp4_kv_read(cache, slots) -> k, v bf16 [T, kv_heads, head_dim]
  nvfp4_kv_attention(q, cache, page_table, seq_lens, prefix=None) -> [B, T, H, D]
"""
import ctypes
import math
import os
from collections import namedtuple

import torch

from . import Fp4qError, _build, _check, _dev, _p, _same_device, _sized, _stream

__all__ = ["rollout_lib", "nvfp4_linear", "mxfp4_linear", "NvFp4KvCache", "nvfp4_kv_cache",
           "nvfp4_kv_append", "nvfp4_kv_read", "nvfp4_kv_attention"]

_lib = None


def declare(L):
    """Argument and result types of every call on a loaded library."""
    vp, i64, ci, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    cache = [vp] * 6 + [i64] * 4
    L.nvfp4_linear.argtypes = [vp, i64, vp, vp, vp, i64, i64, vp, i64, ci, vp, vp, i64, vp]
    L.mxfp4_linear.argtypes = [vp, i64, vp, vp, i64, i64, vp, i64, ci, vp, vp, i64, vp]
    L.nvfp4_kv_append.argtypes = cache + [vp, i64, vp, i64, i64, vp, ci, vp]
    L.nvfp4_kv_read.argtypes = cache + [vp, i64, vp, vp, vp]
    L.nvfp4_kv_attention.argtypes = cache + [vp, i64, i64, i64, i64, vp, i64, vp, vp, i64, vp, vp,
                                             i64, f32, vp, vp, vp, i64, vp]
    for name in ("nvfp4_linear", "mxfp4_linear", "nvfp4_kv_append", "nvfp4_kv_read",
                 "nvfp4_kv_attention"):
        getattr(L, name).restype = ci
    L.nvfp4_linear_workspace_bytes.argtypes = [i64] * 4
    L.mxfp4_linear_workspace_bytes.argtypes = [i64] * 4
    L.nvfp4_kv_attention_workspace_bytes.argtypes = [i64] * 9
    for name in ("nvfp4_linear_workspace_bytes", "mxfp4_linear_workspace_bytes",
                 "nvfp4_kv_attention_workspace_bytes"):
        getattr(L, name).restype = i64
    return L


def rollout_lib():
    """The loaded libfp4q_rollout.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_build.ROLLOUT_PATH):
            raise Fp4qError(
                "libfp4q_rollout.so is not built (%s); run __graft_entry__.build() or "
                "python fp4_block_quantization_amd/_build.py" % _build.ROLLOUT_PATH)
        _lib = declare(ctypes.CDLL(_build.ROLLOUT_PATH))
    return _lib


def _workspace(workspace, need, like):
    """The scratch a call needs: the caller's uint8 tensor, or a new one."""
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=like.device) if need else None
    _dev(workspace, "workspace", torch.uint8)
    if workspace.numel() < need:
        raise Fp4qError("workspace must hold at least %d bytes, got %d"
                        % (need, workspace.numel()))
    return workspace


def _linear(name, mx, x, codes, scales, row_scales, offsets, out_dtype, out, workspace):
    _dev(x, "x", torch.bfloat16)
    _dev(codes, "codes", torch.uint8)
    if x.dim() != 2:
        raise Fp4qError("x must be 2-D [rows, k]")
    if codes.dim() != (2 if offsets is None else 3):
        raise Fp4qError("codes must be [n, k/2], or [groups, n, k/2] with offsets")
    groups = 0 if offsets is None else codes.shape[0]
    rows, k = x.shape
    n = codes.shape[-2]
    if codes.shape[-1] * 2 != k:
        raise Fp4qError("codes hold k = %d, x has %d" % (codes.shape[-1] * 2, k))
    matrices = max(1, groups)
    _sized(scales, "scales", torch.uint8, matrices * n * (k // (32 if mx else 16)))
    if not mx:
        _sized(row_scales, "row_scales", torch.float32, matrices * n)
    if offsets is not None:
        _sized(offsets, "offsets", torch.int64, groups + 1)
    if out is None:
        out = torch.empty((rows, n), dtype=out_dtype, device=x.device)
    if out.dtype not in (torch.bfloat16, torch.float32):
        raise Fp4qError("out must be bfloat16 or float32, got %s" % out.dtype)
    _sized(out, "out", out.dtype, rows * n)
    L = rollout_lib()
    need = getattr(L, name + "_workspace_bytes")(rows, n, k, groups)
    ws = _workspace(workspace, need, x)
    _same_device(x, codes, scales, row_scales, offsets, out, ws)
    tail = (n, k, _p(offsets), groups, int(out.dtype == torch.float32), _p(out), _p(ws),
            0 if ws is None else ws.numel(), _stream(x))
    if mx:
        st = L.mxfp4_linear(_p(x), rows, _p(codes), _p(scales), *tail)
    else:
        st = L.nvfp4_linear(_p(x), rows, _p(codes), _p(scales), _p(row_scales), *tail)
    _check(st, name)
    return out


def nvfp4_linear(x, codes, block_scales, row_scales, offsets=None, out_dtype=torch.bfloat16,
                 out=None, workspace=None):
    """x . DQ(W)^T of a BF16 [rows, k] tensor with NVFP4 weights as
    nvfp4_quantize returns them for W [n, k].  With offsets (int64 GPU tensor
    [experts + 1]) the weights are [experts, n, ..] and rows
    [offsets[e], offsets[e+1]) go through expert e's; other rows of the
    output are not written.  out: optional bfloat16 or float32 [rows, n]."""
    return _linear("nvfp4_linear", False, x, codes, block_scales, row_scales, offsets, out_dtype,
                   out, workspace)


def mxfp4_linear(x, codes, scales, offsets=None, out_dtype=torch.bfloat16, out=None,
                 workspace=None):
    """x . DQ(W)^T with MXFP4 weights (the primary codes and scales of
    mxfp4_resq_quantize); otherwise as nvfp4_linear."""
    return _linear("mxfp4_linear", True, x, codes, scales, None, offsets, out_dtype, out,
                   workspace)


NvFp4KvCache = namedtuple("NvFp4KvCache", "k_codes k_scales k_token_scales "
                                          "v_codes v_scales v_token_scales")
NvFp4KvCache.__doc__ = """A paged NVFP4 key/value cache: k_codes, v_codes u8
[pages, kv_heads, page_size, d/2]; k_scales u8 [pages, kv_heads, page_size,
d/16]; v_scales u8 [pages, kv_heads, d/16, page_size]; k_token_scales,
v_token_scales f32 [pages, kv_heads, page_size].  Token slot p * page_size + o
is place o of page p."""


def nvfp4_kv_cache(num_pages, page_size, kv_heads, head_dim, device="cuda"):
    """A zeroed cache (zeros stand for zero rows)."""
    def make(dtype, *shape):
        return torch.zeros((num_pages, kv_heads) + shape, dtype=dtype, device=device)
    return NvFp4KvCache(make(torch.uint8, page_size, head_dim // 2),
                        make(torch.uint8, page_size, head_dim // 16),
                        make(torch.float32, page_size),
                        make(torch.uint8, page_size, head_dim // 2),
                        make(torch.uint8, head_dim // 16, page_size),
                        make(torch.float32, page_size))


def _cache_args(cache):
    """The six pointers and four sizes of a cache, checked against each other."""
    if len(cache) != 6:
        raise Fp4qError("cache must be an NvFp4KvCache, or its six tensors in order")
    kc = _dev(cache[0], "k_codes", torch.uint8)
    if kc.dim() != 4:
        raise Fp4qError("k_codes must be 4-D [pages, kv_heads, page_size, head_dim/2]")
    pages, heads, page, half = kc.shape
    rows = pages * heads * page
    _sized(cache[1], "k_scales", torch.uint8, rows * (half // 8))
    _sized(cache[2], "k_token_scales", torch.float32, rows)
    _sized(cache[3], "v_codes", torch.uint8, rows * half)
    _sized(cache[4], "v_scales", torch.uint8, rows * (half // 8))
    _sized(cache[5], "v_token_scales", torch.float32, rows)
    return [t.data_ptr() for t in cache] + [pages, page, heads, 2 * half]


def _token_rows(t, name, heads, dim):
    """Token stride of a BF16 [..., heads, dim] tensor whose leading
    dimensions step evenly and whose last two are dense."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise Fp4qError("%s must be a GPU tensor" % name)
    if t.dtype != torch.bfloat16:
        raise Fp4qError("%s must be %s, got %s" % (name, torch.bfloat16, t.dtype))
    if t.dim() < 3 or t.shape[-2] != heads or t.shape[-1] != dim:
        raise Fp4qError("%s must be [..., %d, %d], got %s" % (name, heads, dim, tuple(t.shape)))
    if t.is_contiguous():
        return heads * dim
    stride = t.stride(-3) if t.shape[-3] > 1 else heads * dim
    if (dim > 1 and t.stride(-1) != 1) or (heads > 1 and t.stride(-2) != dim):
        raise Fp4qError("%s must be dense over its last two dimensions" % name)
    step, size = stride, t.shape[-3]
    for i in range(t.dim() - 4, -1, -1):
        if t.shape[i] > 1:
            if size == 1:  # no token step seen yet: this dimension sets it
                stride = step = t.stride(i)
            elif t.stride(i) != step * size:
                raise Fp4qError("%s must step evenly from token to token" % name)
        size *= t.shape[i]
    return stride


def nvfp4_kv_append(cache, k, v, slots, four_over_six=True):
    """Quantize BF16 k and v [tokens, kv_heads, head_dim] into the cache's
    slots (int64 GPU tensor [tokens]; negative: skipped).  Token rows may be
    strided, as slices of a fused projection are."""
    args = _cache_args(cache)
    _, _, heads, dim = args[6:]
    ks, vs = _token_rows(k, "k", heads, dim), _token_rows(v, "v", heads, dim)
    tokens = k.numel() // (heads * dim)
    if v.numel() != k.numel():
        raise Fp4qError("k and v must hold the same tokens")
    _sized(slots, "slots", torch.int64, tokens)
    _same_device(k, v, slots, *cache)
    st = rollout_lib().nvfp4_kv_append(*args, k.data_ptr(), ks, v.data_ptr(), vs, tokens,
                                       slots.data_ptr(), int(four_over_six), _stream(k))
    _check(st, "nvfp4_kv_append")


def nvfp4_kv_read(cache, slots, out=None):
    """BF16 (k, v), each [tokens, kv_heads, head_dim], of the cache's slots
    (int64 GPU tensor [tokens]; a slot outside the cache reads as zeros)."""
    args = _cache_args(cache)
    _, _, heads, dim = args[6:]
    _dev(slots, "slots", torch.int64)
    tokens = slots.numel()
    if out is None:
        out = tuple(torch.empty((tokens, heads, dim), dtype=torch.bfloat16, device=slots.device)
                    for _ in range(2))
    k, v = out
    _sized(k, "k", torch.bfloat16, tokens * heads * dim)
    _sized(v, "v", torch.bfloat16, tokens * heads * dim)
    _same_device(slots, k, v, *cache)
    st = rollout_lib().nvfp4_kv_read(*args, slots.data_ptr(), tokens, k.data_ptr(), v.data_ptr(),
                                     _stream(slots))
    _check(st, "nvfp4_kv_read")
    return k, v


def nvfp4_kv_attention(q, cache, page_table, seq_lens, scale=None, prefix=None, lse=False,
                       out=None, workspace=None):
    """Softmax attention of BF16 q [batch, tokens, heads, head_dim] (or
    [batch, heads, head_dim]) over the cache.  page_table int32 [batch,
    max_pages] and seq_lens int32 [batch] give each sequence's own tokens, the
    queries being its last ones (each sees the tokens up to itself).  prefix:
    optional (prefix_table int32 [groups, pages], prefix_lens int32 [groups],
    group_offsets int32 [groups + 1]): sequences [group_offsets[g],
    group_offsets[g+1]) share prefix g in front of their own tokens; it is
    read once for all of them.  scale: default 1/sqrt(head_dim).  lse=True
    returns (out, log-sum-exp f32) as well."""
    args = _cache_args(cache)
    page, heads, dim = args[7:]
    if not isinstance(q, torch.Tensor) or q.dim() not in (3, 4):
        raise Fp4qError("q must be [batch, tokens, heads, head_dim] or [batch, heads, head_dim]")
    q_heads = q.shape[-2]
    q_stride = _token_rows(q, "q", q_heads, dim)
    batch, tokens = q.shape[0], q.shape[1] if q.dim() == 4 else 1
    _dev(page_table, "page_table", torch.int32)
    if page_table.dim() != 2 or page_table.shape[0] != batch:
        raise Fp4qError("page_table must be [batch, max_pages]")
    _sized(seq_lens, "seq_lens", torch.int32, batch)
    table = lens = offsets = None
    groups = prefix_pages = 0
    if prefix is not None:
        table, lens, offsets = prefix
        _dev(table, "prefix_table", torch.int32)
        if table.dim() != 2 or table.shape[0] == 0:
            raise Fp4qError("prefix_table must be [groups, pages] with at least one group")
        groups, prefix_pages = table.shape
        _sized(lens, "prefix_lens", torch.int32, groups)
        _sized(offsets, "group_offsets", torch.int32, groups + 1)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    _sized(out, "out", torch.bfloat16, q.numel())
    log_sum = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device) if lse else None
    L = rollout_lib()
    need = L.nvfp4_kv_attention_workspace_bytes(page, heads, dim, batch, tokens, q_heads,
                                                page_table.shape[1], prefix_pages, groups)
    ws = _workspace(workspace, need, q)
    _same_device(q, page_table, seq_lens, table, lens, offsets, out, ws, *cache)
    st = L.nvfp4_kv_attention(*args, q.data_ptr(), q_stride, batch, tokens, q_heads,
                              page_table.data_ptr(), page_table.shape[1], seq_lens.data_ptr(),
                              _p(table), prefix_pages, _p(lens), _p(offsets), groups,
                              1.0 / math.sqrt(dim) if scale is None else scale, out.data_ptr(),
                              _p(log_sum), _p(ws), 0 if ws is None else ws.numel(), _stream(q))
    _check(st, "nvfp4_kv_attention")
    return (out, log_sum) if lse else out
