"""The decode step's operators between the products: norm, rotary append, paged attention.

Like the products, these functions pass pointers, sizes and the current CUDA stream to the C ABI in
``include/nvfp4_gemv.h``; there is no other path. They are called many times per token on rows of
a few kilobytes, so their checks and marshalling are native too (``csrc/decode_ops_binding.cpp``).

The cache: ``k_cache`` and ``v_cache`` [pages, kv_heads, page_size, head_dim] (bfloat16, or
float8_e4m3fn with float32 scales per kv head), contiguous inside a page (``kv_cache`` makes a
pair). ``page_table`` int32 [seqs, max_pages] names each sequence's pages in order.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import math
import os
import struct
import threading
from typing import NamedTuple, Optional

import torch

import nvfp4_weight_only_gemv_gb300 as _nv

from . import build as _build

_F32, _BF16, _E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn

# the C structs nvfp4_rms_norm_args, nvfp4_rope_append_args and nvfp4_paged_attention_args as bytes, for
# the C entry points called through the ctypes library (the tests of their checks do)
_NORM = struct.Struct("@6P4q7if").pack
_APPEND = struct.Struct("@14P9q13i2f4x").pack
_ATTEND = struct.Struct("@10P6q10if4x").pack


class _Unbound:
    """Stands in for the native binding until the first call loads the library."""

    def __getattr__(self, name):
        return getattr(_load(), name)


def _load():
    """Loads the binding and gives it the loaded library's entry points."""
    global _native
    with _load_lock:
        if isinstance(_native, _Unbound):  # else another thread was first
            _native = _bound()
        return _native


def _bound():
    lib = _nv.library()
    path = _build.binding_path()
    try:
        _build.build_binding()
    except RuntimeError:  # as for the library: one that is only older than its source serves
        if not os.path.exists(path):
            raise
    loader = importlib.machinery.ExtensionFileLoader("_decode_ops", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_decode_ops", path, loader=loader))
    loader.exec_module(module)
    module.bind(*(ctypes.cast(f, ctypes.c_void_p).value
                  for f in (lib.nvfp4_rms_norm, lib.nvfp4_rope_append, lib.nvfp4_paged_attention)))
    return module


_native = _Unbound()
_load_lock = threading.Lock()


class RMSNormOut(NamedTuple):
    """What rms_norm wrote: the normed rows, the new residual stream and the 8-bit scales."""
    y: torch.Tensor
    residual: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]


def _handle(stream):
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _like(t, name, dtype, shape=None):
    """A new tensor of t's shape (or `shape`) and device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    return torch.empty(t.shape if shape is None else shape, dtype=dtype, device=t.device)


def rms_norm(x, weight, eps: float = 1e-6, residual=None, residual_out=None, out=None, out_dtype=torch.bfloat16,
             scales=None, group: int = 0, stream=None) -> RMSNormOut:
    """y = h / sqrt(mean(h^2) + eps) * weight with h = x + residual, rows of x [rows, cols].

    x, residual and weight are float32 or bfloat16 each; the sum is formed in fp32 and
    ``residual_out`` (new unless given; may be ``residual`` itself) receives it in the residual's
    type. ``out`` (or ``out_dtype``) is float32, bfloat16 or float8_e4m3fn; 8-bit rows come with
    float32 ``scales`` [rows, 1], or [rows, cols / group] for ``group`` columns each (a power of two,
    16 to 256). Rows may be strided. Returns RMSNormOut(y, residual, scales)."""
    if stream is not None and (out is None or (residual is not None and residual_out is None) or
                               (scales is None and getattr(out, "dtype", None) is _E4M3)):
        return _nv._on_stream(stream, rms_norm, x, weight, eps, residual, residual_out, out, out_dtype, scales, group)
    if out is None:
        out = _like(x, "x", out_dtype)
    if residual_out is None and residual is not None:
        residual_out = _like(x, "x", getattr(residual, "dtype", None))
    if scales is None and getattr(out, "dtype", None) is _E4M3:
        scales = _like(x, "x", _F32, (out.shape[0], out.shape[-1] // group if group else 1))
    if stream is not None:
        stream = _handle(stream)
    st = _native.rms_norm(x, weight, eps, residual, residual_out, out, scales, group, stream)
    if st:
        raise _nv.NVFP4Error(st, "nvfp4_rms_norm")
    return RMSNormOut(out, residual_out, scales)


def kv_cache(pages: int, kv_heads: int, page_size: int, head_dim: int, dtype=torch.bfloat16, device=None):
    """A zeroed pair of caches (k, v), each [pages, kv_heads, page_size, head_dim], halves of one
    allocation in which a page's keys and values are neighbours."""
    if dtype not in (_BF16, _E4M3):
        raise TypeError(f"a cache is bfloat16 or float8_e4m3fn (got {dtype})")
    both = torch.zeros((pages, 2, kv_heads, page_size, head_dim), dtype=dtype, device=device or "cuda")
    return both[:, 0], both[:, 1]


def rope_frequencies(rotary_dim: int, base: float = 10000.0, factor: float = 1.0, original_length: int = 0,
                     beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """Rotary frequencies float32 [rotary_dim / 2] and the factor of cos and sin, for rope_append.

    inv_freq[i] = base^(-2 i / rotary_dim). ``factor`` > 1 stretches positions for contexts longer
    than the ``original_length`` trained on: without original_length every frequency is divided by
    it; with it, only frequencies that turn fewer than ``beta_slow`` times over the original length
    are, those above ``beta_fast`` turns stay, the ones between are blended along their index, and
    cos and sin grow by 0.1 ln(factor) + 1 (Peng et al., "YaRN", 2023). Any other rule: pass your
    own inv_freq."""
    if rotary_dim <= 0 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and positive")
    i = torch.arange(rotary_dim // 2, dtype=torch.float64)
    freq = base ** (-2 * i / rotary_dim)
    mscale = 1.0
    if factor > 1.0 and not original_length:
        freq = freq / factor
    elif factor > 1.0:
        def index_of(turns):
            return rotary_dim * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))

        low = max(math.floor(index_of(beta_fast)), 0)
        high = min(math.ceil(index_of(beta_slow)), rotary_dim - 1)
        stretch = ((i - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
        freq = freq / factor * stretch + freq * (1 - stretch)
        mscale = 0.1 * math.log(factor) + 1.0
    return freq.float().to(device or "cuda"), mscale


def rope_append(q, k, v, positions, inv_freq, k_cache, v_cache, page_table, seq_ids=None, *, interleaved: bool = False,
                mscale: float = 1.0, q_norm=None, k_norm=None, eps: float = 1e-6, k_scale=None, v_scale=None,
                out=None, stream=None):
    """Turns q [tokens, q_heads, D] and k by their rotary positions and appends k and v
    [tokens, kv_heads, D] to the cache; returns the turned q as bfloat16 [tokens, q_heads, D]
    (None for q = None).

    q, k, v are all float32 or all bfloat16 and may be views of one fused projection. positions
    int32 [tokens] and seq_ids int32 [tokens] (None: the tokens of each sequence in turn, equally
    many) say where each token stands; a negative position is padding. inv_freq float32 [half]
    turns the first 2 * half values of a head, in halves or ``interleaved`` pairs; mscale multiplies
    cos and sin (rope_frequencies gives both). q_norm, k_norm [D]: root-mean-square norm of each
    head first. k_scale, v_scale float32 [kv_heads]: what an 8-bit cache's values are divided by."""
    if stream is not None and out is None:
        return _nv._on_stream(stream, rope_append, q, k, v, positions, inv_freq, k_cache, v_cache, page_table, seq_ids,
                              interleaved=interleaved, mscale=mscale, q_norm=q_norm, k_norm=k_norm, eps=eps,
                              k_scale=k_scale, v_scale=v_scale)
    if out is None and q is not None:
        out = _like(q, "q", _BF16)
    if stream is not None:
        stream = _handle(stream)
    st = _native.rope_append(q, k, v, positions, inv_freq, k_cache, v_cache, page_table, seq_ids, interleaved, mscale,
                             q_norm, k_norm, eps, k_scale, v_scale, out, stream)
    if st:
        raise _nv.NVFP4Error(st, "nvfp4_rope_append")
    return out


def attention_workspace_bytes(seqs: int, rows: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    """Bytes of workspace paged_attention needs for these sizes, whatever the lengths."""
    n = int(_nv.library().nvfp4_attention_workspace_bytes(seqs, rows, q_heads, kv_heads, head_dim))
    if n < 0:
        raise ValueError(f"no attention workspace for seqs={seqs}, rows={rows}, heads={q_heads}/{kv_heads}, D={head_dim}")
    return n


def attention_workspace(seqs: int, rows: int, q_heads: int, kv_heads: int, head_dim: int, device=None) -> torch.Tensor:
    """A zeroed workspace for paged_attention (uint8). Reuse it, also for other sizes that need no more
    bytes: every call leaves its counters at zero. Calls that share one must be ordered."""
    n = attention_workspace_bytes(seqs, rows, q_heads, kv_heads, head_dim)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def _workspace_for(q, k_cache, page_table):
    """A workspace for one call; the smallest there is where the call will be refused anyway."""
    try:
        seqs = page_table.shape[0]
        n = attention_workspace_bytes(seqs, q.shape[0] // seqs if seqs else 0, q.shape[1], k_cache.shape[1], q.shape[2])
    except (AttributeError, IndexError, ValueError):
        n = 256
    return torch.zeros(n, dtype=torch.uint8, device=q.device)


def paged_attention(q, k_cache, v_cache, page_table, lengths, scale: Optional[float] = None, *, window: int = 0,
                    k_scale=None, v_scale=None, workspace=None, out=None, lse=None, stream=None):
    """softmax(scale * q . k) v over the cached keys, for the newest tokens of each sequence.

    q bfloat16 [seqs * rows, q_heads, D] holds the newest ``rows`` (1 to 8) tokens of each sequence,
    the rows of a sequence together; lengths int32 [seqs] counts each sequence's cached tokens, these
    included. Row r sees the keys up to its own position, lengths - rows + r, and with ``window``
    only the last ``window`` of them. q_heads is a multiple of the cache's kv heads. scale: 1 /
    sqrt(D) unless given. ``lse``: an optional float32 [seqs * rows, q_heads] tensor that receives
    the log of each row's sum of exponentials. ``workspace``: a uint8 tensor zeroed before its first
    use, of at least attention_workspace_bytes; None allocates one for this call. Returns bfloat16
    like q; rows that see no key are zero (lse -inf)."""
    if stream is not None and (out is None or workspace is None):
        return _nv._on_stream(stream, paged_attention, q, k_cache, v_cache, page_table, lengths, scale, window=window,
                              k_scale=k_scale, v_scale=v_scale, workspace=workspace, out=out, lse=lse)
    if out is None:
        out = _like(q, "q", _BF16)
    if workspace is None:
        workspace = _workspace_for(q, k_cache, page_table)
    if stream is not None:
        stream = _handle(stream)
    st = _native.paged_attention(q, k_cache, v_cache, page_table, lengths, q.shape[-1] ** -0.5 if scale is None else scale,
                                 window, k_scale, v_scale, workspace, out, lse, stream)
    if st:
        raise _nv.NVFP4Error(st, "nvfp4_paged_attention")
    return out
