"""A paged cache of keys and values, and the operators that fill and read it.

Pages are shared by all sequences; a page table gives each sequence its pages in
order.  The cache holds the inputs' type, or 8-bit e4m3 codes with one fp32 scale
for each (page, head).  The work runs in libtriattn.so's kernels.
"""
from __future__ import annotations

import math
from typing import Optional

import torch

from . import abi
from .api import _DT, _check_out, _int32, _need, _on, _ptr, _row_stride, _stream
from .positions import Rotary, _check_rotary

_CACHE_DT = {**_DT, torch.float8_e4m3fn: abi.TA_E4M3}


class PagedKVCache:
    """The pages of a cache: k and v (num_pages, Hk, page_size, D), with k_scale and v_scale
    (num_pages, Hk) float32 where they hold float8_e4m3fn codes (an element stands for code * scale;
    v_scale from 2^-56 to 2^56).

    The tensors are used in place.  k and v may be strided views whose last
    dimension is contiguous, such as the halves of one (num_pages, 2, Hk,
    page_size, D) buffer or a (num_pages, page_size, Hk, D) buffer with its middle
    dimensions exchanged.  page_size is a power of two from 16 to 1024.
    """

    def __init__(self, k, v, k_scale=None, v_scale=None):
        for t, nm in ((k, "k"), (v, "v")):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{nm} must be a torch.Tensor")
            if t.dim() != 4:
                raise ValueError(f"{nm} must be (num_pages, Hk, page_size, D)")
            if t.dtype not in _CACHE_DT:
                raise TypeError("the cache must be float32, float16, bfloat16 or float8_e4m3fn")
            if t.stride(3) != 1:
                raise ValueError(f"{nm}: the last dimension (D) must be contiguous")
        if v.shape != k.shape or v.dtype != k.dtype or v.device != k.device:
            raise ValueError("k and v must share shape, dtype and device")
        self.num_pages, self.heads, self.page_size, self.head_dim = k.shape
        self.dtype, self.device = k.dtype, k.device
        if k.dtype == torch.float8_e4m3fn:
            for t, nm in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                _need(t, nm, k.device)
                if t.dtype != torch.float32 or tuple(t.shape) != (self.num_pages, self.heads):
                    raise ValueError(f"{nm} must be float32 {(self.num_pages, self.heads)}")
        elif k_scale is not None or v_scale is not None:
            raise ValueError("scales belong to a float8_e4m3fn cache")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self._code = _CACHE_DT[k.dtype]
        self._strides = tuple(None if t.is_contiguous() else
                              abi.strides3([t.stride(i) if t.shape[i] > 1 else t.shape[2] * t.shape[3] * t.shape[1]
                                            for i in range(3)]) for t in (k, v))

    @classmethod
    def empty(cls, num_pages, heads, page_size, head_dim, dtype=torch.bfloat16, device="cuda"):
        """A new cache; its memory is not initialised (rows are written before they are read)."""
        k, v = (torch.empty(num_pages, heads, page_size, head_dim, dtype=dtype, device=device) for _ in range(2))
        ks = vs = None
        if dtype == torch.float8_e4m3fn:
            ks, vs = (torch.zeros(num_pages, heads, dtype=torch.float32, device=device) for _ in range(2))
        return cls(k, v, ks, vs)


def _table(page_table, kv_lengths, cu_seqlens, dev):
    """(number of sequences, pages a sequence) of the three int32 tensors that describe the sequences."""
    for t, nm in ((page_table, "page_table"), (kv_lengths, "kv_lengths")):
        _need(t, nm, dev)
        if t.dtype != torch.int32:
            raise TypeError(f"{nm} must be int32")
    if page_table.dim() != 2:
        raise ValueError("page_table must be (num_seqs, max_pages)")
    S, MP = page_table.shape
    if kv_lengths.numel() != S:
        raise ValueError("kv_lengths must have one entry per row of page_table")
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", dev)
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.numel() != S + 1:
            raise ValueError("cu_seqlens must be int32 with num_seqs + 1 entries")
    return S, MP


def _rows(t, name, dev, dtype, total, D):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 3 or t.shape[0] != total or t.shape[2] != D:
        raise ValueError(f"{name} must be (total, H, D) with total = {total}, D = {D}")
    if t.dtype != dtype:
        raise TypeError("q, k and v must share one dtype")
    return _row_stride(t, name, dev)


def kv_cache_append(cache: PagedKVCache, k, v, page_table, kv_lengths, cu_seqlens=None, max_seqlen=1, *,
                    rotary: Optional[Rotary] = None, positions=None, q=None, out_q=None):
    """Writes the new rows k, v (total, Hk, D) of each sequence into the cache, in place.

    cu_seqlens (S + 1,) int32 splits the rows over the sequences (at most
    max_seqlen each; none is fine; rows past its last entry are left alone); without it
    row i belongs to sequence i.  kv_lengths (S,) int32 counts the slots that a
    sequence holds after this call: the new rows are the last of them.
    page_table (S, max_pages) int32; a page that is written has one place in the
    tables of the call.  rotary turns k, and q (total, Hq, D) if given, by each row's slot or
    by positions (total,) int32.  Returns the turned q (out_q, which may be q), or None.

    An 8-bit cache takes a power-of-two scale for each (page, head): rows that need
    a larger one re-code the rows before them.  It starts anew with the row in slot 0 of the page and does not
    shrink when rows are written over.  Infinities and NaN become NaN.
    """
    if not isinstance(cache, PagedKVCache):
        raise TypeError("cache must be a PagedKVCache")
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("expected k (total, Hk, D)")
    dev = k.device
    if dev.type != "cuda":
        raise ValueError("kv_cache_append runs on CUDA tensors only")
    if cache.device != dev:
        raise ValueError(f"cache is on {cache.device}, expected {dev}")
    if k.dtype not in _DT:
        raise TypeError("k must be float32, float16 or bfloat16")
    total, Hk, D = k.shape
    if Hk != cache.heads or D != cache.head_dim:
        raise ValueError(f"k must have the cache's {cache.heads} heads of {cache.head_dim}")
    k_rs, v_rs = _rows(k, "k", dev, k.dtype, total, D), _rows(v, "v", dev, k.dtype, total, D)
    if v.shape[1] != Hk:
        raise ValueError("v must have k's heads")
    S, MP = _table(page_table, kv_lengths, cu_seqlens, dev)
    max_seqlen = int(max_seqlen)
    if cu_seqlens is None and (total != S or max_seqlen != 1):
        raise ValueError("without cu_seqlens there is one row for each sequence")
    Hq = q_rs = qo_rs = 0
    if q is not None:
        if rotary is None:
            raise ValueError("q is given only to be turned: pass rotary")
        q_rs, Hq = _rows(q, "q", dev, k.dtype, total, D), q.shape[1]
        if out_q is None:
            out_q, qo_rs = torch.empty(q.shape, dtype=q.dtype, device=dev), Hq * D
        else:
            qo_rs = _rows(out_q, "out_q", dev, k.dtype, total, D)
            if out_q.shape != q.shape:
                raise ValueError("out_q must have q's shape")
    elif out_q is not None:
        raise ValueError("out_q needs q")
    if positions is not None:
        if rotary is None:
            raise ValueError("positions need rotary")
        _need(positions, "positions", dev)
        if positions.dtype != torch.int32 or positions.numel() != total:
            raise ValueError("positions must be int32 with one entry per row")
    turns, dim, inter, ms = 0, 0, False, 1.0
    if rotary is not None:
        _check_rotary(rotary, dev)
        turns, dim, inter, ms = _ptr(rotary.turns), rotary.dim, rotary.interleaved, rotary.attention_factor
    if total == 0 or S == 0:
        return out_q
    with _on(dev):
        abi.tri_attn_kv_append(_ptr(q), _ptr(k), _ptr(v), _DT[k.dtype], _ptr(cu_seqlens), _ptr(kv_lengths),
                               _ptr(page_table), S, total, max_seqlen, Hq, Hk, D, q_rs, k_rs, v_rs, qo_rs,
                               _ptr(positions), turns, dim, inter, ms, _ptr(cache.k), _ptr(cache.v), cache._code,
                               _ptr(cache.k_scale), _ptr(cache.v_scale), cache.num_pages, cache.page_size, MP,
                               cache._strides[0], cache._strides[1], _ptr(out_q), _stream(dev))
    return out_q


def paged_attention(q, cache: PagedKVCache, page_table, kv_lengths, cu_seqlens_q=None, max_seqlen_q=1, scale=None, *,
                    window=None, sinks=0, return_aux=False, out=None):
    """Attention of each sequence's newest tokens over its pages of the cache.

    q (total_q, Hq, D), Hq a multiple of the cache's heads (consecutive query heads
    share one).  kv_lengths (S,) int32 counts the slots a sequence holds, its rows of q
    among them: row j of n sees the slots up to kv_lengths - n + j.
    cu_seqlens_q (S + 1,) int32 splits the rows (at most max_seqlen_q each; rows past its
    last entry are left alone); without it there is one row for each sequence.
    window: only the last ``window`` of those slots, and the first ``sinks`` of the
    sequence.  scale defaults to 1/sqrt(D).  Returns O, or (O, lse) with return_aux (lse
    float32 (Hq, total_q)); a row that sees no slot gets O = 0 and lse = -inf.

    Made for few new tokens a sequence: K and V are read again for each 16 rows (tokens x query heads
    of a key head).  A whole prompt without a cached prefix runs faster through ``varlen_attention``
    (which takes as many heads of k and v as of q).
    """
    if not isinstance(cache, PagedKVCache):
        raise TypeError("cache must be a PagedKVCache")
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    if q.dim() != 3:
        raise ValueError("expected q (total_q, Hq, D)")
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("paged_attention runs on CUDA tensors only")
    if cache.device != dev:
        raise ValueError(f"cache is on {cache.device}, expected {dev}")
    if q.dtype not in _DT:
        raise TypeError("q must be float32, float16 or bfloat16")
    total, Hq, D = q.shape
    Hk = cache.heads
    if D != cache.head_dim:
        raise ValueError(f"q must have the cache's head dimension {cache.head_dim}")
    if Hk == 0 or Hq % Hk:
        raise ValueError(f"q's heads must be a multiple of the cache's {Hk}")
    q_rs = _row_stride(q, "q", dev)
    S, MP = _table(page_table, kv_lengths, cu_seqlens_q, dev)
    max_seqlen_q = int(max_seqlen_q)
    if cu_seqlens_q is None and (total != S or max_seqlen_q != 1):
        raise ValueError("without cu_seqlens_q there is one row for each sequence")
    if window is not None and int(window) < 1:
        raise ValueError("window must be at least 1")
    if int(sinks) < 0:
        raise ValueError("sinks must not be negative")
    s = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    else:
        _check_out(out, q.shape, q.dtype)
        _need(out, "out", dev)
    lse = torch.empty(Hq, total, dtype=torch.float32, device=dev) if return_aux else None
    if total and S:
        code = _DT[q.dtype]
        nbytes = abi.tri_attn_paged_workspace_size(code, max_seqlen_q, Hq, Hk, D)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        with _on(dev):
            abi.tri_attn_paged_fwd(_ptr(q), code, _ptr(cu_seqlens_q), _ptr(kv_lengths), _ptr(page_table), S, total,
                                   max_seqlen_q, Hq, Hk, D, q_rs, s, 0 if window is None else _int32(window), _int32(sinks),
                                   _ptr(cache.k), _ptr(cache.v), cache._code, _ptr(cache.k_scale), _ptr(cache.v_scale),
                                   cache.num_pages, cache.page_size, MP, cache._strides[0], cache._strides[1],
                                   _ptr(out), _ptr(lse), _ptr(ws), nbytes, _stream(dev))
    return (out, lse) if return_aux else out
