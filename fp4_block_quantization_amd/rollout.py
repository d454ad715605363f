"""Operators of a 4-bit rollout engine -- Python binding of
libfp4q_rollout.so (C ABI in include/fp4q/rollout.h).

Argument marshalling only, in the manner of the package's other calls: GPU
tensors in, outputs allocated on the inputs' device or passed in, launches
on torch's current stream, no CPU fallback.  The checks are in a native
module (csrc_rollout/rollout_ext.cpp): in Python they took longer than the
smaller kernels run.  There is no backward pass: in grad mode an input that
requires a gradient is refused.

  nvfp4_linear(x, codes, block_scales, row_scales, offsets=None) -> [R, N]
  mxfp4_linear(x, codes, scales, offsets=None) -> [R, N]
  nvfp4_kv_cache(num_pages, page_size, kv_heads, head_dim) -> NvFp4KvCache
  nvfp4_kv_append(cache, k, v, slots, four_over_six=True)
  nvfp4_kv_read(cache, slots) -> k, v bf16 [T, kv_heads, head_dim]
  nvfp4_kv_attention(q, cache, page_table, seq_lens, prefix=None) -> [B, T, H, D]
"""
import ctypes
import importlib.machinery
import importlib.util
import os
from collections import namedtuple

import torch

from . import Fp4qError, _build, _check, _raw_stream

__all__ = ["rollout_lib", "nvfp4_linear", "mxfp4_linear", "NvFp4KvCache", "nvfp4_kv_cache",
           "nvfp4_kv_append", "nvfp4_kv_read", "nvfp4_kv_attention"]

_lib = None
_ext = None


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


def _open(path, what):
    if not os.path.exists(path):
        raise Fp4qError("%s is not built (%s); run __graft_entry__.build() or "
                        "python fp4_block_quantization_amd/_build.py" % (what, path))
    return path


def rollout_lib():
    """The loaded libfp4q_rollout.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        _lib = declare(ctypes.CDLL(_open(_build.ROLLOUT_PATH, "libfp4q_rollout.so")))
    return _lib


def _current_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


def _native_module(name, path):
    """A native half of the binding, loaded from the in-tree build."""
    loader = importlib.machinery.ExtensionFileLoader(name, _open(path, name + ".so"))
    spec = importlib.util.spec_from_file_location(name, path, loader=loader)
    ext = importlib.util.module_from_spec(spec)
    loader.exec_module(ext)
    return ext


def _native():
    """The native half of this binding, its calls bound to the library's."""
    global _ext
    if _ext is None:
        ext = _native_module("fp4q_rollout_ext", _build.ROLLOUT_EXT_PATH)
        bind(ext, rollout_lib())
        _ext = ext
    return _ext


def bind(ext, L):
    """Hand a loaded library's entry points to the native half."""
    calls = (L.nvfp4_linear, L.nvfp4_linear_workspace_bytes, L.mxfp4_linear,
             L.mxfp4_linear_workspace_bytes, L.nvfp4_kv_append, L.nvfp4_kv_read,
             L.nvfp4_kv_attention, L.nvfp4_kv_attention_workspace_bytes)
    ext.bind(Fp4qError, _check, _raw_stream or _current_stream,
             *[ctypes.cast(c, ctypes.c_void_p).value for c in calls])


def _fp32(out_dtype, out):
    if out is not None:
        if out_dtype is not None and out_dtype is not getattr(out, "dtype", None):
            raise Fp4qError("out is not of out_dtype %s" % (out_dtype,))
        return False  # out's own type decides
    if out_dtype is None or out_dtype is torch.bfloat16:
        return False
    if out_dtype is torch.float32:
        return True
    raise Fp4qError("out_dtype must be torch.bfloat16 or torch.float32, got %s" % (out_dtype,))


def nvfp4_linear(x, codes, block_scales, row_scales, offsets=None, out_dtype=None, out=None,
                 workspace=None):
    """x . DQ(W)^T of a BF16 [rows, k] tensor with NVFP4 weights as
    nvfp4_quantize returns them for W [n, k]: codes [n, k/2], block_scales
    [n, k/16], row_scales [n].  With offsets (int64 GPU tensor [experts + 1])
    each is [experts, n, ..] and rows [offsets[e], offsets[e+1]) go through
    expert e's; other rows of the output are not written.  out_dtype:
    bfloat16 (default) or float32; out: optional [rows, n] of either, whose
    type decides.  Tensors of another shape are refused, also
    where they hold as many elements."""
    return (_ext or _native()).linear(False, x, codes, block_scales, row_scales, offsets,
                                      _fp32(out_dtype, out), out, workspace)


def mxfp4_linear(x, codes, scales, offsets=None, out_dtype=None, out=None, workspace=None):
    """x . DQ(W)^T with MXFP4 weights (the primary codes and scales of
    mxfp4_resq_quantize); otherwise as nvfp4_linear."""
    return (_ext or _native()).linear(True, x, codes, scales, None, offsets,
                                      _fp32(out_dtype, out), out, workspace)


NvFp4KvCache = namedtuple("NvFp4KvCache", "k_codes k_scales k_token_scales "
                                          "v_codes v_scales v_token_scales")
NvFp4KvCache.__doc__ = """A paged NVFP4 key/value cache: k_codes, v_codes u8
[pages, kv_heads, page_size, d/2] (d a multiple of 16; attention takes 64,
128, 192 and 256); k_scales u8 [pages, kv_heads, page_size,
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


def nvfp4_kv_append(cache, k, v, slots, four_over_six=True):
    """Quantize BF16 k and v [tokens, kv_heads, head_dim] into the cache's
    slots (int64 GPU tensor [tokens]; negative: skipped).  Token rows may be
    strided, as slices of a fused projection are."""
    (_ext or _native()).append(cache, k, v, slots, int(four_over_six))


def nvfp4_kv_read(cache, slots, out=None):
    """BF16 (k, v), each [tokens, kv_heads, head_dim], of the cache's slots
    (int64 GPU tensor [tokens]; a slot outside the cache reads as zeros)."""
    return (_ext or _native()).read(cache, slots, out)


def nvfp4_kv_attention(q, cache, page_table, seq_lens, scale=None, prefix=None, lse=False,
                       out=None, workspace=None):
    """Softmax attention of BF16 q [batch, tokens, heads, head_dim] (or
    [batch, heads, head_dim]) over the cache.  page_table int32 [batch,
    max_pages] and seq_lens int32 [batch] give each sequence's own tokens, the
    queries being its last ones (each sees the tokens up to itself).  prefix:
    optional (prefix_table int32 [groups, pages], prefix_lens int32 [groups],
    group_offsets int32 [groups + 1]): sequences [group_offsets[g],
    group_offsets[g+1]) share prefix g in front of their own tokens; it is
    read and decoded once per 16 (groups of more than 256 query rows a cache
    head: 32) of those rows.  scale: default 1/sqrt(head_dim).  head_dim 64,
    128, 192 or 256.  lse=True returns (out, log-sum-exp f32) as well."""
    return (_ext or _native()).attention(q, cache, page_table, seq_lens, scale, prefix, lse, out,
                                         workspace)
