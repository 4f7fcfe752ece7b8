"""Binding of the paged-cache operators (``include/dit_paged.h``).

* ``dit_rope_frequencies``           pair frequencies, scaled for long contexts
* ``dit_qk_rope_scaled``             optional per-head RMSNorm and rotary positions from such a table
* ``dit_qkv_rope_append``            the same on the way into a paged cache, v beside it
* ``dit_paged_attention``            attention of a chunk of new tokens over the cache
* ``dit_paged_attention_workspace``  bytes of workspace it wants

A call runs on its tensors' device (all on one) and on ``stream``, by default
that device's current stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import Optional, Sequence

import torch

from . import _call, _packing, _rows

_ROPE_MODES = {"interleaved": 0, "half": 1, "none": 2}
_ROPE_SCALES = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


def _one_device(first: torch.Tensor, *others) -> int:
    """The CUDA device all the tensors lie on (None stands for an absent one)."""
    index = first.get_device()
    if index < 0:
        raise ValueError("expected CUDA tensors")
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError(f"all tensors must lie on one device, got {first.device} and {t.device}")
    return index


def _stream_on(index: int, stream) -> int:
    """The raw stream a call runs on: the device's current one, or the given."""
    if stream is None:
        return torch.cuda.current_stream(index).cuda_stream if _raw_stream is None else _raw_stream(index)
    if isinstance(stream, torch.cuda.Stream):
        if stream.device_index != index:
            raise ValueError(f"the stream belongs to {stream.device}, the tensors to cuda:{index}")
        return stream.cuda_stream
    return int(stream)


def _allocating_stream(index: int, on: int, stream) -> torch.cuda.Stream:
    """The stream that owns what a call on ``stream`` (raw: ``on``) allocates.
    Raw 0 and 1 are the default stream; torch.cuda.ExternalStream takes a 0 for
    no stream given and hands out one of its own pool, on which memory would be
    reused while the call still runs."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(on, device=index) if on > 1 else torch.cuda.default_stream(index)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call_on(index: int, name: str, *args) -> None:
    """The library launches on the current device; make it the tensors'."""
    if _raw_device() == index:
        _call(name, *args)
    else:
        with torch.cuda.device(index):
            _call(name, *args)


def _pack(cu_seqlens: torch.Tensor, cu_seqlens_padded: torch.Tensor) -> tuple:
    n = cu_seqlens.shape
    if cu_seqlens_padded is cu_seqlens and cu_seqlens.dtype is torch.int32 and len(n) == 1 and n[0] > 0 and \
            cu_seqlens.is_contiguous():  # nothing is padded
        p = cu_seqlens.data_ptr()
        return p, p, n[0] - 1
    if cu_seqlens.dtype is torch.int32 and cu_seqlens_padded.dtype is torch.int32 and len(n) == 1 and n[0] > 0 and \
            cu_seqlens_padded.shape == n and cu_seqlens.is_contiguous() and cu_seqlens_padded.is_contiguous():
        return cu_seqlens.data_ptr(), cu_seqlens_padded.data_ptr(), n[0] - 1
    return _packing(cu_seqlens, cu_seqlens_padded)  # says what is wrong


def _ints(t: torch.Tensor, shape: tuple, what: str) -> int:
    if t.dtype is not torch.int32 or t.shape != shape or not t.is_contiguous():
        raise TypeError(f"{what}: expected a contiguous int32 CUDA tensor {list(shape)}")
    return t.data_ptr() or None


def _freqs(t: torch.Tensor, n: Optional[int], what: str) -> int:
    shape = t.shape
    if t.dtype is not torch.float64 or len(shape) != 1 or not t.is_contiguous() or (n is not None and shape[0] != n):
        raise TypeError(f"{what}: expected a contiguous float64 CUDA vector"
                        + ("" if n is None else f" of {n} entries"))
    return t.data_ptr()


def _heads(t: torch.Tensor, heads: int, head_dim: int, rows: int, what: str) -> tuple:
    """(pointer, row stride) of [rows, heads * head_dim] or [rows, heads, head_dim]."""
    width = heads * head_dim
    if t.dtype is torch.bfloat16 and t.shape == (rows, width):  # the usual case, first
        if width == 0:
            return None, 0
        st = t.stride()
        if st[1] == 1:
            return t.data_ptr(), st[0] if rows > 1 else width
    ptr, stride = _rows(t, what)
    if t.size(0) != rows or t.numel() != rows * heads * head_dim:
        raise ValueError(f"{what}: expected {rows} rows of {heads} heads of {head_dim}, got {tuple(t.shape)}")
    # one row has no stride of its own: torch may report any
    return ptr, stride if rows > 1 else heads * head_dim


def _cache_strides(st: tuple, pages: int, page_size: int, heads: int, head_dim: int) -> tuple:
    """An axis of one entry has no stride: any multiple of 8 does."""
    return (st[0] if pages > 1 else page_size * heads * head_dim,
            st[1] if page_size > 1 else max(head_dim, st[1] // 8 * 8),
            st[2] if heads > 1 else head_dim, 1)


def _cache(k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor, heads: int, head_dim: int,
           B: int) -> tuple:
    shape = k_cache.shape
    if k_cache.dtype is not torch.bfloat16 or v_cache.dtype is not torch.bfloat16:
        raise TypeError("k_cache, v_cache: expected bfloat16 CUDA tensors")
    if len(shape) != 4 or shape[2] != heads or shape[3] != head_dim or v_cache.shape != shape:
        raise ValueError(f"k_cache, v_cache: expected [pages, page_size, {heads}, {head_dim}], got {tuple(shape)} and "
                         f"{tuple(v_cache.shape)}")
    pages, page_size = shape[0], shape[1]
    ks, vs = k_cache.stride(), v_cache.stride()
    if ks[3] != 1 or vs[3] != 1:
        raise ValueError("k_cache, v_cache: the last axis must be contiguous")

    if pages == 1 or page_size == 1 or heads == 1:
        ks, vs = (_cache_strides(st, pages, page_size, heads, head_dim) for st in (ks, vs))
    if ks != vs:
        raise ValueError("k_cache and v_cache must have the same strides")
    ts, tt = block_table.shape, block_table.stride()
    if block_table.dtype is not torch.int32 or len(ts) != 2 or ts[0] != B or (ts[1] > 1 and tt[1] != 1):
        raise TypeError("block_table: expected an int32 CUDA tensor [num_seqs, max_pages], contiguous rows")
    table_stride = tt[0] if B > 1 else ts[1]
    return (k_cache.data_ptr() or None, v_cache.data_ptr() or None, ks[0], ks[1], ks[2], pages, page_size), \
        (block_table.data_ptr() or None, table_stride, ts[1])


def dit_rope_frequencies(rotary_dim: int, *, theta: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                         original_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                         device="cuda") -> tuple:
    """(freqs, attn_scale): float64 [rotary_dim / 2] on ``device`` and the
    factor on cos and sin.  scaling: "none", "linear", "ntk" or "yarn" (see the
    header for the formulas; yarn reads original_len and the betas).  Build it
    once and keep it; tables of grid sections are concatenated."""
    table = (ctypes.c_double * max(1, rotary_dim // 2))()
    gain = ctypes.c_float()
    _call("dit_rope_frequencies", rotary_dim, float(theta), _ROPE_SCALES[scaling], float(factor), int(original_len),
          float(beta_fast), float(beta_slow), table, ctypes.byref(gain))
    return torch.tensor(list(table), dtype=torch.float64, device=device), gain.value


def _rope_args(freqs, rope_grid, grid_freqs, sections, pos_offset, attn_scale, eps, rope_mode, B):
    mode = _ROPE_MODES[rope_mode]
    st, sh, sw = (int(s) for s in sections)
    fp = gp = gf = None
    rotary = 0
    if mode != 2:
        if freqs is None:
            raise TypeError("freqs: expected a frequency table (dit_rope_frequencies)")
        fp, rotary = _freqs(freqs, None, "freqs"), 2 * freqs.numel()
        if rope_grid is not None:
            gp = _ints(rope_grid, (B, 3), "rope_grid")
            if grid_freqs is None:
                raise TypeError("grid_freqs: needed with rope_grid")
            gf = _freqs(grid_freqs, freqs.numel(), "grid_freqs")
    po = None if pos_offset is None else _ints(pos_offset, (B,), "pos_offset")
    return fp, rotary, gp, gf, st, sh, sw, po, float(attn_scale), float(eps), mode


def _weights(q_weight, k_weight, head_dim):
    if (q_weight is None) != (k_weight is None):
        raise ValueError("give both norm weights or neither")
    if q_weight is None:
        return None, None
    for t, what in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if t.dtype is not torch.bfloat16:
            raise TypeError(f"{what}: expected bfloat16, got {t.dtype}")
        if t.numel() != head_dim or not t.is_contiguous():
            raise ValueError(f"{what}: expected a contiguous vector of {head_dim}")
    return q_weight.data_ptr(), k_weight.data_ptr()


def dit_qk_rope_scaled(q: torch.Tensor, k: torch.Tensor, cu_seqlens: torch.Tensor, cu_seqlens_padded: torch.Tensor,
                       *, num_q_heads: int, num_k_heads: int, head_dim: int, freqs: Optional[torch.Tensor],
                       q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                       rope_grid: Optional[torch.Tensor] = None, grid_freqs: Optional[torch.Tensor] = None,
                       sections: Sequence[int] = (0, 0, 0), pos_offset: Optional[torch.Tensor] = None,
                       attn_scale: float = 1.0, eps: float = 1e-6, rope_mode: str = "interleaved",
                       q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                       stream=None) -> tuple:
    """q_out, k_out <- rotation by p * freqs of the first 2 * len(freqs)
    elements of every head of q and k, behind the per-head RMSNorm when both
    weights are given.  Without q_out / k_out in place.  Row r of sequence b
    has position pos_offset[b] + r (0 without offsets); with rope_grid
    (int32 [num_seqs, 3]) rows inside the grid turn by their t, h, w
    coordinates times grid_freqs over ``sections``.  rope_mode: "interleaved",
    "half" or "none".  Returns (q_out, k_out)."""
    qo, ko = q if q_out is None else q_out, k if k_out is None else k_out
    dev = _one_device(q, k, qo, ko, cu_seqlens, cu_seqlens_padded, freqs, q_weight, k_weight, rope_grid, grid_freqs,
                      pos_offset)
    rows = q.size(0)
    qp, qs = _heads(q, num_q_heads, head_dim, rows, "q")
    kp, ks = _heads(k, num_k_heads, head_dim, rows, "k")
    qop, qos = _heads(qo, num_q_heads, head_dim, rows, "q_out")
    kop, kos = _heads(ko, num_k_heads, head_dim, rows, "k_out")
    cs, cp, B = _pack(cu_seqlens, cu_seqlens_padded)
    wq, wk = _weights(q_weight, k_weight, head_dim)
    fp, rotary, gp, gf, st, sh, sw, po, gain, eps, mode = _rope_args(
        freqs, rope_grid, grid_freqs, sections, pos_offset, attn_scale, eps, rope_mode, B)
    _call_on(dev, "dit_qk_rope_scaled", qp, qs, kp, ks, qop, qos, kop, kos, wq, wk, cs, cp, B, rows, num_q_heads,
             num_k_heads, head_dim, fp, rotary, gp, gf, st, sh, sw, po, gain, eps, mode, _stream_on(dev, stream))
    return qo, ko


def dit_qkv_rope_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor,
                        v_cache: torch.Tensor, block_table: torch.Tensor, cache_lens: torch.Tensor,
                        cu_seqlens: torch.Tensor, cu_seqlens_padded: torch.Tensor, *, num_q_heads: int,
                        num_kv_heads: int, head_dim: int, freqs: Optional[torch.Tensor],
                        q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                        rope_grid: Optional[torch.Tensor] = None, grid_freqs: Optional[torch.Tensor] = None,
                        sections: Sequence[int] = (0, 0, 0), pos_offset: Optional[torch.Tensor] = None,
                        attn_scale: float = 1.0, eps: float = 1e-6, rope_mode: str = "interleaved",
                        q_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dit_qk_rope_scaled on the way into a paged cache: q to q_out (or in
    place), k into its slots of k_cache, v copied into those of v_cache; k and
    v are only read.  k_cache, v_cache: bf16 [pages, page_size, num_kv_heads,
    head_dim] of any (equal) strides over the first three axes; block_table:
    int32 [num_seqs, max_pages]; cache_lens: int32 [num_seqs], the tokens
    cached before this call (not advanced).  pos_offset: positions of the first
    rows, by default cache_lens.  Returns q_out."""
    qo = q if q_out is None else q_out
    dev = _one_device(q, k, v, qo, k_cache, v_cache, block_table, cache_lens, cu_seqlens, cu_seqlens_padded, freqs,
                      q_weight, k_weight, rope_grid, grid_freqs, pos_offset)
    rows = q.size(0)
    qp, qs = _heads(q, num_q_heads, head_dim, rows, "q")
    kp, ks = _heads(k, num_kv_heads, head_dim, rows, "k")
    vp, vs = _heads(v, num_kv_heads, head_dim, rows, "v")
    qop, qos = _heads(qo, num_q_heads, head_dim, rows, "q_out")
    cs, cp, B = _pack(cu_seqlens, cu_seqlens_padded)
    wq, wk = _weights(q_weight, k_weight, head_dim)
    cache, table = _cache(k_cache, v_cache, block_table, num_kv_heads, head_dim, B)
    fp, rotary, gp, gf, st, sh, sw, po, gain, eps, mode = _rope_args(
        freqs, rope_grid, grid_freqs, sections, pos_offset, attn_scale, eps, rope_mode, B)
    _call_on(dev, "dit_qkv_rope_append", qp, qs, kp, ks, vp, vs, qop, qos, wq, wk, *cache, *table,
             _ints(cache_lens, (B,), "cache_lens"), cs, cp, B, rows, num_q_heads, num_kv_heads, head_dim, fp, rotary,
             gp, gf, st, sh, sw, po, gain, eps, mode, _stream_on(dev, stream))
    return qo


def dit_paged_attention_workspace(num_rows_padded: int, num_seqs: int, *, num_q_heads: int, num_kv_heads: int,
                                  head_dim: int, max_kv_len: int, max_chunk: int = 0) -> int:
    """Bytes of workspace dit_paged_attention wants for these sizes (it may be
    0).  max_kv_len: what the call passes, or the table's capacity."""
    n = ctypes.c_int64()
    _call("dit_paged_attention_workspace", num_rows_padded, num_seqs, num_q_heads, num_kv_heads, head_dim, max_chunk,
          max_kv_len, ctypes.byref(n))
    return n.value


def dit_paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                        kv_lens: torch.Tensor, cu_seqlens: torch.Tensor, cu_seqlens_padded: torch.Tensor, *,
                        num_q_heads: int, num_kv_heads: int, head_dim: int, softmax_scale: Optional[float] = None,
                        causal: bool = True, window: int = 0, max_chunk: int = 0, max_kv_len: int = 0,
                        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of each sequence's new tokens over its kv_lens[b] cached
    tokens, the last of which are the new ones (dit_qkv_rope_append first).

    q: bf16 [rows, num_q_heads * head_dim], any row stride; caches and table as
    in dit_qkv_rope_append.  causal: a token sees itself and what lies before
    it, else everything cached; window > 0: only tokens j > p - window.
    softmax_scale: 1 / sqrt(head_dim) by default.  max_chunk, max_kv_len: the
    batch's longest chunk and kv_lens where the host knows them (they choose
    kernels, never the result).  lse: fp32 [rows, num_q_heads] to fill, or None.
    workspace: uint8 CUDA tensor of dit_paged_attention_workspace bytes, one per
    call in flight; None allocates it.  Returns out, whose padding rows are
    left as they are (uninitialised when out is None)."""
    rows = q.size(0)
    dev = _one_device(q, k_cache, v_cache, block_table, kv_lens, cu_seqlens, cu_seqlens_padded, out, lse, workspace)
    qp, qs = _heads(q, num_q_heads, head_dim, rows, "q")
    cs, cp, B = _pack(cu_seqlens, cu_seqlens_padded)
    cache, table = _cache(k_cache, v_cache, block_table, num_kv_heads, head_dim, B)
    lens = _ints(kv_lens, (B,), "kv_lens")
    if lse is not None and (lse.dtype != torch.float32 or not lse.is_cuda or not lse.is_contiguous()
                            or tuple(lse.shape) != (rows, num_q_heads)):
        raise TypeError(f"lse: expected a contiguous float32 CUDA tensor [{rows}, {num_q_heads}]")
    if workspace is not None and (workspace.dtype != torch.uint8 or not workspace.is_contiguous()):
        raise TypeError("workspace: expected a contiguous uint8 CUDA tensor")
    if not 0 <= window < 2**31:
        raise ValueError("window: expected 0 (none) or a number of tokens below 2**31")
    scale = 1.0 / math.sqrt(head_dim) if softmax_scale is None else float(softmax_scale)
    on = _stream_on(dev, stream)
    if out is None or (workspace is None and rows > 0 and B > 0):
        # what is allocated here belongs to the stream that uses it
        with torch.cuda.device(dev), (contextlib.nullcontext() if stream is None else
                                      torch.cuda.stream(_allocating_stream(dev, on, stream))):
            if out is None:
                out = torch.empty((rows, num_q_heads * head_dim), dtype=q.dtype, device=q.device)
            if workspace is None:
                capacity = max(1, min(table[2] * cache[6], 2**31 - 1))
                workspace = torch.empty(dit_paged_attention_workspace(
                    rows, B, num_q_heads=num_q_heads, num_kv_heads=num_kv_heads, head_dim=head_dim,
                    max_chunk=max_chunk, max_kv_len=min(max_kv_len, capacity) if max_kv_len > 0 else capacity),
                    dtype=torch.uint8, device=q.device)
    op, os_ = _heads(out, num_q_heads, head_dim, rows, "out")
    nbytes = 0 if workspace is None else workspace.numel()
    _call_on(dev, "dit_paged_attention", qp, qs, *cache, *table, lens, cs, cp, B, rows, num_q_heads, num_kv_heads,
             head_dim, scale, int(bool(causal)), int(window), int(max_chunk), int(max_kv_len), op, os_,
             None if lse is None else lse.data_ptr(), workspace.data_ptr() if nbytes else None, nbytes, on)
    return out
