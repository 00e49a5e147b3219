"""The decode step's operators between the products: norm, rotary append, paged attention.

Like the products, every function here checks tensors and passes pointers, sizes and the current
CUDA stream to the C ABI in ``include/nvfp4_gemv.h``; there is no other path. These calls are made
many times per token on rows of a few kilobytes, so the checks are kept short and the arguments go
over as one packed struct.

The cache: ``k_cache`` and ``v_cache`` [pages, kv_heads, page_size, head_dim] (bfloat16, or
float8_e4m3fn with float32 scales per kv head), contiguous inside a page (``kv_cache`` makes a
pair). ``page_table`` int32 [seqs, max_pages] names each sequence's pages in order.
"""
from __future__ import annotations

import math
import struct
from typing import NamedTuple, Optional

import torch

import nvfp4_weight_only_gemv_gb300 as _nv

_F32, _BF16, _E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
_CODE = {_F32: 0, _BF16: 1, _E4M3: 2}
_WIDE = (_F32, _BF16)
_CACHE = (_BF16, _E4M3)

# the C structs nvfp4_rms_norm_args, nvfp4_rope_append_args and nvfp4_paged_attention_args
_NORM = struct.Struct("@6P4q7if").pack
_APPEND = struct.Struct("@14P9q13i2f4x").pack
_ATTEND = struct.Struct("@10P6q10if4x").pack

_raw_stream = torch._C._cuda_getCurrentRawStream


def _device() -> int:
    """The current CUDA device; -2, which no tensor is on, where there is none."""
    try:
        return torch._C._cuda_getDevice()
    except RuntimeError:
        return -2


class RMSNormOut(NamedTuple):
    """What rms_norm wrote: the normed rows, the new residual stream and the 8-bit scales."""
    y: torch.Tensor
    residual: Optional[torch.Tensor]
    scales: Optional[torch.Tensor]


def _stream(stream, dev):
    if stream is None:
        return _raw_stream(dev)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _bad(t, name, dtypes, ndim, dev):
    """The error for a tensor that _check turned down."""
    if not isinstance(t, torch.Tensor):
        return TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        return ValueError(f"{name} must be a CUDA tensor (got {t.device})")
    if t.dtype not in dtypes:
        return TypeError(f"{name} must be {' or '.join(map(str, dtypes))} (got {t.dtype})")
    if t.dim() != ndim:
        return ValueError(f"{name} must have {ndim} dims (got {tuple(t.shape)})")
    if t.get_device() != dev:
        return ValueError(f"every tensor must be on the current CUDA device cuda:{dev} (got {t.device})")
    return ValueError(f"{name} must have unit stride in its last dimension (got strides {t.stride()})")


def _check(t, name, dtypes, ndim, dev):
    if (not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.dim() != ndim or t.get_device() != dev
            or (t.stride(-1) != 1 and t.shape[-1] > 1)):
        raise _bad(t, name, dtypes, ndim, dev)


def _contiguous(t, name, dtypes, ndim, dev):
    _check(t, name, dtypes, ndim, dev)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def rms_norm(x, weight, eps: float = 1e-6, residual=None, residual_out=None, out=None, out_dtype=torch.bfloat16,
             scales=None, group: int = 0, stream=None) -> RMSNormOut:
    """y = h / sqrt(mean(h^2) + eps) * weight with h = x + residual, rows of x [rows, cols].

    x, residual and weight are float32 or bfloat16 each; the sum is formed in fp32 and
    ``residual_out`` (new unless given; may be ``residual`` itself) receives it in the residual's
    type. ``out`` (or ``out_dtype``) is float32, bfloat16 or float8_e4m3fn; 8-bit rows come with
    float32 ``scales`` [rows, 1], or [rows, cols / group] for ``group`` columns each (a power of two,
    16 to 256). Rows may be strided. Returns RMSNormOut(y, residual, scales)."""
    dev = _device()
    _check(x, "x", _WIDE, 2, dev)
    _check(weight, "weight", _WIDE, 1, dev)
    rows, cols = x.shape
    if weight.shape[0] != cols:
        raise ValueError(f"weight must have {cols} values (got {weight.shape[0]})")
    if out is None:
        out = torch.empty((rows, cols), dtype=out_dtype, device=x.device)
    _check(out, "out", (_F32, _BF16, _E4M3), 2, dev)
    if out.shape != x.shape:
        raise ValueError(f"out must have shape {tuple(x.shape)} (got {tuple(out.shape)})")
    rp = rop = sp = ldr = ldro = rt = 0
    if residual is not None:
        _check(residual, "residual", _WIDE, 2, dev)
        if residual_out is None:
            residual_out = torch.empty((rows, cols), dtype=residual.dtype, device=x.device)
        _check(residual_out, "residual_out", (residual.dtype,), 2, dev)
        if residual.shape != x.shape or residual_out.shape != x.shape:
            raise ValueError(f"residual and residual_out must have shape {tuple(x.shape)}")
        rp, rop, ldr, ldro, rt = (residual.data_ptr(), residual_out.data_ptr(), residual.stride(0),
                                  residual_out.stride(0), _CODE[residual.dtype])
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    if out.dtype is _E4M3:
        if group and cols % group:
            raise ValueError(f"group {group} does not divide {cols} columns")
        shape = (rows, cols // group if group else 1)
        if scales is None:
            scales = torch.empty(shape, dtype=_F32, device=x.device)
        _contiguous(scales, "scales", (_F32,), 2, dev)
        if tuple(scales.shape) != shape:
            raise ValueError(f"scales must have shape {shape} (got {tuple(scales.shape)})")
        sp = scales.data_ptr()
    elif scales is not None or group:
        raise ValueError("scales and group belong to a float8_e4m3fn output")
    st = _nv.library().nvfp4_rms_norm(
        _NORM(x.data_ptr(), rp, weight.data_ptr(), rop, out.data_ptr(), sp, x.stride(0), ldr, ldro, out.stride(0),
              _CODE[x.dtype], rt, _CODE[weight.dtype], _CODE[out.dtype], rows, cols, group, eps), _stream(stream, dev))
    if st:
        raise _nv.NVFP4Error(st, "nvfp4_rms_norm")
    return RMSNormOut(out, residual_out, scales)


def kv_cache(pages: int, kv_heads: int, page_size: int, head_dim: int, dtype=torch.bfloat16, device=None):
    """A zeroed pair of caches (k, v), each [pages, kv_heads, page_size, head_dim], halves of one
    allocation in which a page's keys and values are neighbours."""
    if dtype not in _CACHE:
        raise TypeError(f"a cache is bfloat16 or float8_e4m3fn (got {dtype})")
    both = torch.zeros((pages, 2, kv_heads, page_size, head_dim), dtype=dtype, device=device or "cuda")
    return both[:, 0], both[:, 1]


def _check_cache(k_cache, v_cache, dev):
    _check(k_cache, "k_cache", _CACHE, 4, dev)
    _check(v_cache, "v_cache", (k_cache.dtype,), 4, dev)
    if v_cache.shape != k_cache.shape:
        raise ValueError(f"k_cache {tuple(k_cache.shape)} and v_cache {tuple(v_cache.shape)} differ")
    _, heads, page, dim = k_cache.shape
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if t.stride()[1:] != (page * dim, dim, 1) and t.numel() and not t[0].is_contiguous():
            raise ValueError(f"{name} must be contiguous inside a page (got strides {t.stride()})")


def _head_scale(t, name, heads, dev):
    if t is None:
        return 0
    _contiguous(t, name, (_F32,), 1, dev)
    if t.shape[0] != heads:
        raise ValueError(f"{name} must have one value per kv head ({heads}, got {t.shape[0]})")
    return t.data_ptr()


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
    dev = _device()
    _check(k, "k", _WIDE, 3, dev)
    same = (k.dtype,)
    _check(v, "v", same, 3, dev)
    _check_cache(k_cache, v_cache, dev)
    _contiguous(positions, "positions", (torch.int32,), 1, dev)
    _contiguous(inv_freq, "inv_freq", (_F32,), 1, dev)
    _check(page_table, "page_table", (torch.int32,), 2, dev)
    tokens, kv_heads, dim = k.shape
    pages, cache_heads, page, cache_dim = k_cache.shape
    if v.shape != k.shape or cache_heads != kv_heads or cache_dim != dim or positions.shape[0] != tokens:
        raise ValueError(f"shape mismatch: k {tuple(k.shape)}, v {tuple(v.shape)}, cache {tuple(k_cache.shape)}, "
                         f"positions {tuple(positions.shape)}")
    half = inv_freq.shape[0]
    if 2 * half > dim:
        raise ValueError(f"inv_freq turns {2 * half} values of a head of {dim}")
    seqs, max_pages = page_table.shape
    sid = 0
    if seq_ids is not None:
        _contiguous(seq_ids, "seq_ids", (torch.int32,), 1, dev)
        if seq_ids.shape[0] != tokens:
            raise ValueError(f"seq_ids must have {tokens} values (got {seq_ids.shape[0]})")
        sid = seq_ids.data_ptr()
    elif seqs == 0 or tokens % seqs:
        raise ValueError(f"{tokens} tokens do not divide among {seqs} sequences: pass seq_ids")
    norms = [0, 0]
    norm_type = 0
    for i, (w, name) in enumerate(((q_norm, "q_norm"), (k_norm, "k_norm"))):
        if w is not None:
            _contiguous(w, name, _WIDE, 1, dev)
            if w.shape[0] != dim or (norms[0] and w.dtype != q_norm.dtype):
                raise ValueError("q_norm and k_norm must have head_dim values of one type")
            norms[i], norm_type = w.data_ptr(), _CODE[w.dtype]
    qp = op = q_heads = qt = qh = 0
    if q is not None:
        _check(q, "q", same, 3, dev)
        q_heads = q.shape[1]
        if q.shape[0] != tokens or q.shape[2] != dim:
            raise ValueError(f"q must be [{tokens}, heads, {dim}] (got {tuple(q.shape)})")
        if out is None:
            out = torch.empty(q.shape, dtype=_BF16, device=q.device)
        _contiguous(out, "out", (_BF16,), 3, dev)
        if out.shape != q.shape:
            raise ValueError(f"out must have shape {tuple(q.shape)} (got {tuple(out.shape)})")
        qp, op, qt, qh = q.data_ptr(), out.data_ptr(), q.stride(0), q.stride(1)
    elif out is not None or q_norm is not None:
        raise ValueError("out and q_norm belong to q")
    st = _nv.library().nvfp4_rope_append(
        _APPEND(qp, k.data_ptr(), v.data_ptr(), positions.data_ptr(), sid, inv_freq.data_ptr(), norms[0], norms[1],
                op, k_cache.data_ptr(), v_cache.data_ptr(), _head_scale(k_scale, "k_scale", kv_heads, dev),
                _head_scale(v_scale, "v_scale", kv_heads, dev), page_table.data_ptr(),
                qt, qh, k.stride(0), k.stride(1), v.stride(0), v.stride(1), k_cache.stride(0), v_cache.stride(0),
                page_table.stride(0), _CODE[k.dtype], norm_type, _CODE[k_cache.dtype], tokens, seqs, q_heads, kv_heads,
                dim, half, interleaved, pages, max_pages, page, mscale, eps), _stream(stream, dev))
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
    """A zeroed workspace for paged_attention (uint8). Reuse it: every call leaves its counters at
    zero. Calls that share one must be ordered."""
    n = attention_workspace_bytes(seqs, rows, q_heads, kv_heads, head_dim)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


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
    dev = _device()
    _check(q, "q", (_BF16,), 3, dev)
    _check_cache(k_cache, v_cache, dev)
    _check(page_table, "page_table", (torch.int32,), 2, dev)
    _contiguous(lengths, "lengths", (torch.int32,), 1, dev)
    tokens, q_heads, dim = q.shape
    pages, kv_heads, page, cache_dim = k_cache.shape
    seqs, max_pages = page_table.shape
    if lengths.shape[0] != seqs or cache_dim != dim or (tokens % seqs if seqs else tokens):
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, cache {tuple(k_cache.shape)}, page_table "
                         f"{tuple(page_table.shape)}, lengths {tuple(lengths.shape)}")
    if kv_heads == 0 and q_heads or kv_heads and q_heads % kv_heads:
        raise ValueError(f"{q_heads} query heads do not divide among {kv_heads} kv heads")
    rows = tokens // seqs if seqs else 0
    if workspace is None:
        workspace = attention_workspace(seqs, rows, q_heads, kv_heads, dim, q.device)
    _contiguous(workspace, "workspace", (torch.uint8,), 1, dev)
    if out is None:
        out = torch.empty(q.shape, dtype=_BF16, device=q.device)
    _contiguous(out, "out", (_BF16,), 3, dev)
    if out.shape != q.shape:
        raise ValueError(f"out must have shape {tuple(q.shape)} (got {tuple(out.shape)})")
    lp = 0
    if lse is not None:
        _contiguous(lse, "lse", (_F32,), 2, dev)
        if lse.shape != q.shape[:2]:
            raise ValueError(f"lse must have shape {tuple(q.shape[:2])} (got {tuple(lse.shape)})")
        lp = lse.data_ptr()
    if scale is None:
        scale = dim ** -0.5 if dim else 1.0
    st = _nv.library().nvfp4_paged_attention(
        _ATTEND(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _head_scale(k_scale, "k_scale", kv_heads, dev),
                _head_scale(v_scale, "v_scale", kv_heads, dev), page_table.data_ptr(), lengths.data_ptr(),
                out.data_ptr(), lp, workspace.data_ptr(), q.stride(0), q.stride(1), k_cache.stride(0),
                v_cache.stride(0), page_table.stride(0), workspace.numel(), _CODE[k_cache.dtype], seqs, rows, q_heads,
                kv_heads, dim, pages, max_pages, page, window, scale), _stream(stream, dev))
    if st:
        raise _nv.NVFP4Error(st, "nvfp4_paged_attention")
    return out
