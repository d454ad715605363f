"""The operators between a layer's 4-bit products, cache and attention --
Python binding of libfp4q_rollout.so (C ABI in include/fp4q/layer.h).

In the manner of rollout.py: GPU tensors in, outputs allocated on the inputs'
device or passed in, launches on torch's current stream, checks in a native
module (csrc_rollout/layer_ext.cpp), no CPU fallback, no backward pass (in
grad mode an input that requires a gradient is refused).  An out= must not
overlap an input or another output, but where its call says so.

  rotary_frequencies(dims, base=10000.0, method="none", ..) -> frequencies, amplitude
  rotary(q, k, positions, frequencies, amplitude=1.0) -> q, k
  prompt_attention(q, k, v, q_offsets, k_offsets=None) -> [tokens, H, D]
  moe_route(logits, top_k, ..) -> weights, experts
  moe_dispatch(x, experts, num_experts) -> rows, offsets, place
  moe_combine(y, place, weights, add=None) -> [tokens, n]
"""
import ctypes
import math

import torch

from . import Fp4qError, _build, _check, _raw_stream
from .rollout import _current_stream, _fp32, _native_module, rollout_lib

__all__ = ["rotary_frequencies", "rotary", "prompt_attention", "moe_route", "moe_dispatch",
           "moe_combine"]

_ext = None


def declare(L):
    """Argument and result types of every call on a loaded library."""
    vp, i64, ci, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    L.rotary_embed.argtypes = [vp, i64, i64, vp, i64, i64, i64, i64, i64, vp, vp, f32, ci, ci, ci,
                               vp, i64, vp, i64, vp]
    L.prompt_attention.argtypes = [vp, i64, i64, i64, vp, i64, vp, i64, i64, i64, i64, vp, vp, i64,
                                   f32, vp, vp, vp, i64, vp]
    L.moe_route.argtypes = [vp, ci, i64, i64, i64, vp, ci, i64, i64, ci, f32, vp, vp, vp, vp]
    L.moe_dispatch.argtypes = [vp, i64, i64, vp, i64, i64, vp, vp, vp, vp, i64, vp]
    L.moe_combine.argtypes = [vp, ci, i64, vp, vp, vp, i64, i64, i64, ci, vp, vp]
    for name in ("rotary_embed", "prompt_attention", "moe_route", "moe_dispatch", "moe_combine"):
        getattr(L, name).restype = ci
    L.prompt_attention_workspace_bytes.argtypes = [i64] * 6
    L.moe_dispatch_workspace_bytes.argtypes = [i64] * 3
    for name in ("prompt_attention_workspace_bytes", "moe_dispatch_workspace_bytes"):
        getattr(L, name).restype = i64
    return L


def _native():
    """The native half of this binding, its calls bound to the library's."""
    global _ext
    if _ext is None:
        ext = _native_module("fp4q_layer_ext", _build.LAYER_EXT_PATH)
        L = declare(rollout_lib())
        calls = (L.rotary_embed, L.prompt_attention, L.prompt_attention_workspace_bytes,
                 L.moe_route, L.moe_dispatch, L.moe_dispatch_workspace_bytes, L.moe_combine)
        ext.bind(Fp4qError, _check, _raw_stream or _current_stream,
                 *[ctypes.cast(c, ctypes.c_void_p).value for c in calls])
        _ext = ext
    return _ext


def rotary_frequencies(dims, base=10000.0, method="none", factor=1.0, original_positions=None,
                       slow=1.0, fast=32.0, amplitude=None, device="cuda"):
    """Frequencies (float64 [dims / 2] on device, radians a position: base **
    (-2 i / dims)) and the amplitude that rotary() takes, for contexts
    stretched by factor:

      "none"       as they are
      "positions"  every frequency divided by factor
      "base"       base * factor ** (dims / (dims - 2)): the slowest divided by factor
      "parts"      pairs that turn more than `fast` times within
                   original_positions keep their frequency, those that turn
                   less than `slow` times have it divided by factor, those in
                   between a mixture, linear in the turns; the amplitude is
                   0.1 ln(factor) + 1 unless given

    For other scalings pass rotary() frequencies of your own."""
    if dims < 2 or dims % 2:
        raise Fp4qError("dims must be even and at least 2, got %r" % (dims,))
    if not (0 < base < math.inf and 0 < factor < math.inf):
        raise Fp4qError("base and factor must be positive and finite")
    divided, kept = 1.0, None
    if method == "positions":
        divided = factor
    elif method == "base":
        if dims == 2:
            raise Fp4qError('method "base" needs more than one pair')
    elif method == "parts":
        if original_positions is None or original_positions <= 0 or not slow < fast:
            raise Fp4qError('method "parts" needs original_positions, and slow below fast')
        divided, kept = factor, original_positions / (2.0 * math.pi)
    elif method != "none":
        raise Fp4qError('method must be "none", "positions", "base" or "parts", got %r' % (method,))
    out = []
    try:
        if method == "base":
            base = base * factor ** (dims / (dims - 2.0))
        for i in range(dims // 2):
            f = base ** (-2.0 * i / dims)
            share = 0.0 if kept is None else min(max((f * kept - slow) / (fast - slow), 0.0), 1.0)
            out.append(f * share + f / divided * (1.0 - share))
    except (OverflowError, ZeroDivisionError):
        out = [math.inf]
    if not all(map(math.isfinite, out)):
        raise Fp4qError("these arguments do not give finite frequencies")
    if amplitude is None:
        amplitude = 0.1 * math.log(factor) + 1.0 if method == "parts" else 1.0
    return torch.tensor(out, dtype=torch.float64, device=device), float(amplitude)


def rotary(q, k, positions, frequencies, amplitude=1.0, interleaved=False, inverse=False, out=None):
    """Turn the first 2 * len(frequencies) elements of every head of q and k
    ([.., heads, head_dim], BF16 or FP32; k may be None) by positions (int64
    GPU tensor, one for each token) times frequencies (float64 GPU tensor [dims
    / 2], as rotary_frequencies gives), and scale them by amplitude.  Pairs
    are (i, i + dims / 2), or interleaved (2 i, 2 i + 1).  inverse=True turns
    back.  Rows may be strided, as slices of a fused projection are; out:
    optional (q, k), which may be the inputs themselves.  Returns (q, k)."""
    return (_ext or _native()).rotary(q, k, positions, frequencies, amplitude, interleaved, inverse,
                                      out)


def prompt_attention(q, k, v, q_offsets, k_offsets=None, scale=None, lse=False, out=None,
                     workspace=None):
    """Causal softmax attention of packed BF16 sequences: q [tokens, heads,
    head_dim], k and v [k_tokens, kv_heads, head_dim] (rows may be strided, as
    slices of a fused projection are).  Sequence b has the queries
    [q_offsets[b], q_offsets[b + 1]) and the keys [k_offsets[b], k_offsets[b +
    1]) (int32 GPU tensors [sequences + 1]; k_offsets None: q_offsets); its
    queries are the last of its keys.  So it takes whole prompts, and chunks
    behind a context that nvfp4_kv_read has read back; of a longer buffer of keys
    pass the rows in use, by which long contexts are cut into parts.  scale:
    default 1/sqrt(head_dim).  head_dim 64, 128, 192 or 256.  Rows outside the
    sequences are left as they are (out=).  lse=True returns (out, log-sum-exp
    f32 [tokens, heads]) as well."""
    return (_ext or _native()).prompt(q, k, v, q_offsets, k_offsets, scale, lse, out, workspace)


def moe_route(logits, top_k, bias=None, scoring="softmax", groups=1, top_groups=1,
              renormalize=True, scale=1.0, active=None, out=None):
    """The top_k experts of every token (int32 [tokens, top_k], best first, the
    lower index of equal ones) and their weights (FP32), from BF16 or FP32
    logits [tokens, experts].  Scores are softmax or sigmoid; bias (FP32
    [experts]) is added for the choice only; with groups > 1 only experts of
    the top_groups groups of neighbours with the largest sums of their two best
    can be chosen.  Weights: the chosen scores, with renormalize divided by
    their sum, times scale.  active: optional bool [tokens]; other tokens
    (padding) get the experts -1 and weights 0.  out: optional (weights,
    experts)."""
    if scoring not in ("softmax", "sigmoid"):
        raise Fp4qError('scoring must be "softmax" or "sigmoid", got %r' % (scoring,))
    return (_ext or _native()).route(logits, top_k, bias, scoring == "sigmoid", groups, top_groups,
                                     renormalize, scale, active, out)


def moe_dispatch(x, experts, num_experts, out=None, workspace=None):
    """BF16 x [tokens, hidden] by expert: (rows [tokens * top_k, hidden],
    offsets int64 [num_experts + 1], place int32 [tokens, top_k]) for experts
    as moe_route gives them.  rows[place[t, j]] is x[t]; expert e's rows are
    [offsets[e], offsets[e + 1]), in the tokens' order: what nvfp4_linear and
    mxfp4_linear take as x and offsets.  An expert outside [0, num_experts) gets
    no row and the place -1; rows past the last are left as they are."""
    return (_ext or _native()).dispatch(x, experts, num_experts, out, workspace)


def moe_combine(y, place, weights, add=None, out_dtype=None, out=None):
    """The experts' rows y (BF16 or FP32 [rows, n]) back to their tokens: add[t]
    (BF16 [tokens, n], optional) + the sum over j of weights[t, j] * y[place[t,
    j]], summed in FP32.  A place outside y adds nothing.  out_dtype: bfloat16
    (default) or float32; out: optional [tokens, n] of either, whose type
    decides; a BF16 one may be add."""
    return (_ext or _native()).combine(y, place, weights, add, _fp32(out_dtype, out), out)
