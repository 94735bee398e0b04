"""A paged cache of keys and values, and the operators that fill and read it.

Pages are shared by all sequences; a page table gives each sequence its pages in
order.  The cache holds the inputs' type, 8-bit e4m3 codes with one fp32 scale
for each (page, head), or 4-bit whole numbers with an e4m3 scale for 16 neighbours.  The work runs in libtriattn.so's kernels.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Union

import torch

from . import abi
from .api import _DT, _check_out, _int32, _need, _new, _on, _ptr, _row_stride, _stream
from .positions import Rotary, _check_positions, _check_rotary

_CACHE_DT = {**_DT, torch.float8_e4m3fn: abi.TA_E4M3}


class _Parts:
    """The tensors of a cache as public attributes, and what the calls read of them (`_describe`), made again by `_now` where another
    tensor, or other memory of one, stands there: a call must not use memory that the cache no longer holds."""

    _PARTS = ("k", "v", "k_scale", "v_scale")
    _OWN = ("_c", "_strides", "_at")  # what a copy describes anew

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name in self._PARTS:
            object.__setattr__(self, "_at", None)

    def _renew(self):
        self._describe()
        self._at = tuple([_ptr(getattr(self, n)) for n in self._PARTS])

    # (8-bit floating point as bytes: plain pickle cannot read such tensors back)
    def __getstate__(self):
        state = {n: x for n, x in self.__dict__.items() if n not in self._OWN}
        eight = [n for n in self._PARTS if isinstance(state.get(n), torch.Tensor) and state[n].dtype == torch.float8_e4m3fn]
        return {**state, **{n: state[n].view(torch.uint8) for n in eight}}, eight

    def __setstate__(self, state):
        state, eight = state
        self.__dict__.update({**state, **{n: state[n].view(torch.float8_e4m3fn) for n in eight}, "_at": None})


class PagedKVCache(_Parts):
    """The pages of a cache: k and v (num_pages, Hk, page_size, D), with k_scale and v_scale
    (num_pages, Hk) float32 where they hold float8_e4m3fn codes (an element stands for code * scale;
    v_scale from 2^-56 to 2^56).

    The tensors are used in place, as they are at each call (another may be put in
    one's place).  k and v may be strided views whose last dimension is contiguous,
    such as the halves of one (num_pages, 2, Hk, page_size, D) buffer or a (num_pages,
    page_size, Hk, D) buffer with its middle dimensions exchanged.  page_size is a power of two from 16 to 1024.
    """

    def __init__(self, k, v, k_scale=None, v_scale=None):
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self._now()

    def _now(self):
        if self._at is None or self._at != (self.k.data_ptr(), self.v.data_ptr(), _ptr(self.k_scale), _ptr(self.v_scale)):
            self._renew()

    def _describe(self):
        k, v, k_scale, v_scale = self.k, self.v, self.k_scale, self.v_scale
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


class PagedKVCache4(_Parts):
    """The pages of a 4-bit cache: an element of head h stands for n * scale * factor[h], n a whole number from -7 to 7.

    k, v: uint8 (num_pages, Hk, page_size, D / 2), two codes n + 8 a byte (the even element in the low half);
    k_scale, v_scale: float8_e4m3fn (num_pages, Hk, page_size, D / 16), one for 16 neighbouring elements of a row;
    k_factor, v_factor: float32 (Hk,) or None (1), from 2^-100 to 2^100, fixed for the cache's life (powers of two cost no
    precision; a factor around the 100th part of a head's usual magnitudes keeps its scales in e4m3's middle).

    The tensors are used in place, as they are at each call (another may be put in one's place).  Pages and heads may be
    strided (a head's page is contiguous), such as the halves of one (num_pages, 2, Hk, page_size, D / 2) buffer.  page_size is
    a power of two from 16 to 1024, D a multiple of 32.
    """

    _PARTS = _Parts._PARTS + ("k_factor", "v_factor")

    def __init__(self, k, v, k_scale, v_scale, k_factor=None, v_factor=None):
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.k_factor, self.v_factor = k_factor, v_factor
        self._now()

    def _now(self):
        if self._at is None or self._at != (self.k.data_ptr(), self.v.data_ptr(), self.k_scale.data_ptr(), self.v_scale.data_ptr(),
                                            _ptr(self.k_factor), _ptr(self.v_factor)):
            self._renew()

    def _describe(self):
        k, v, k_scale, v_scale, k_factor, v_factor = (getattr(self, n) for n in self._PARTS)
        for t, nm in ((k, "k"), (v, "v"), (k_scale, "k_scale"), (v_scale, "v_scale")):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{nm} must be a torch.Tensor")
            if t.dim() != 4:
                raise ValueError(f"{nm} must have four dimensions (num_pages, Hk, page_size, ...)")
            want = torch.uint8 if nm in "kv" else torch.float8_e4m3fn
            if t.dtype != want:
                raise TypeError(f"{nm} must be {want}")
            if t.device != k.device:
                raise ValueError(f"{nm} is on {t.device}, expected {k.device}")
            if t.stride(3) != 1 or (t.shape[2] > 1 and t.stride(2) != t.shape[3]):
                raise ValueError(f"{nm}: a head's page (the last two dimensions) must be contiguous")
        self.num_pages, self.heads, self.page_size, half = k.shape
        self.head_dim, self.dtype, self.device = 2 * half, torch.uint8, k.device
        if self.head_dim % 32:
            raise ValueError("the head dimension must be a multiple of 32")
        if v.shape != k.shape:
            raise ValueError("k and v must share their shape")
        for t, nm in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if tuple(t.shape) != (self.num_pages, self.heads, self.page_size, self.head_dim // 16):
                raise ValueError(f"{nm} must be {(self.num_pages, self.heads, self.page_size, self.head_dim // 16)}")
        for t, nm in ((k_factor, "k_factor"), (v_factor, "v_factor")):
            if t is None:
                continue
            _need(t, nm, k.device)
            if t.dtype != torch.float32 or tuple(t.shape) != (self.heads,):
                raise ValueError(f"{nm} must be float32 {(self.heads,)}")
        strides = (ctypes.c_longlong * 8)()
        parts = (k, v, k_scale, v_scale)
        if not all(t.is_contiguous() for t in parts):
            for i, t in enumerate(parts):
                least = t.shape[2] * t.shape[3]
                head = t.stride(1) if t.shape[1] > 1 else least
                strides[2 * i] = t.stride(0) if t.shape[0] > 1 else max(head * t.shape[1], least)
                if head < least or strides[2 * i] < least:  # (an expanded tensor; strides that are all 0 mean a contiguous one)
                    raise ValueError("pages or heads of the cache's tensors overlap")
                strides[2 * i + 1] = head
        self._c = abi.Cache4(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), _ptr(k_factor) or None,
                             _ptr(v_factor) or None, self.num_pages, self.page_size, strides)

    @classmethod
    def empty(cls, num_pages, heads, page_size, head_dim, k_factor=None, v_factor=None, device="cuda"):
        """A new cache; its memory is not initialised (rows are written before they are read)."""
        k, v = (torch.empty(num_pages, heads, page_size, head_dim // 2, dtype=torch.uint8, device=device) for _ in range(2))
        ks, vs = (torch.empty(num_pages, heads, page_size, head_dim // 16, dtype=torch.uint8,
                              device=device).view(torch.float8_e4m3fn) for _ in range(2))
        return cls(k, v, ks, vs, k_factor, v_factor)


_CACHES = (PagedKVCache, PagedKVCache4)


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


def kv_cache_append(cache: Union[PagedKVCache, PagedKVCache4], k, v, page_table, kv_lengths, cu_seqlens=None, max_seqlen=1, *,
                    rotary: Optional[Rotary] = None, positions=None, q=None, out_q=None):
    """Writes the new rows k, v (total, Hk, D) of each sequence into the cache, in place.

    cu_seqlens (S + 1,) int32 splits the rows over the sequences (at most
    max_seqlen each; none is fine; rows past its last entry are left alone); without it
    row i belongs to sequence i.  kv_lengths (S,) int32 counts the slots that a
    sequence holds after this call: the new rows are the last of them.
    page_table (S, max_pages) int32; a page that is written has one place in the
    tables of the call.  rotary turns k, and q (total, Hq, D) if given, by each row's slot or
    by positions (total,) int32 ((axes, total) where rotary has sections; without positions every axis
    is the slot).  Returns the turned q (out_q, which may be q), or None.

    An 8-bit cache takes a power-of-two scale for each (page, head): rows that need
    a larger one re-code the rows before them.  It starts anew with the row in slot 0 of the page and does not
    shrink when rows are written over.  Infinities and NaN become NaN.
    A 4-bit cache takes an e4m3 scale for 16 elements of a row, and rows keep their codes (rotary.dim a multiple of
    32); an infinity or NaN makes its 16 elements NaN.
    """
    if not isinstance(cache, _CACHES):
        raise TypeError("cache must be a PagedKVCache or a PagedKVCache4")
    cache._now()
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("expected k (total, Hk, D)")
    dev = k.device
    if not k.is_cuda:
        raise ValueError("kv_cache_append runs on CUDA tensors only")
    if cache.device != dev:
        raise ValueError(f"cache is on {cache.device}, expected {dev}")
    if k.dtype not in _DT:
        raise TypeError("k must be float32, float16 or bfloat16")
    total, Hk, D = k.shape
    if Hk != cache.heads or D != cache.head_dim:
        raise ValueError(f"k must have the cache's {cache.heads} heads of {cache.head_dim}")
    k_rs, v_rs = _row_stride(k, "k", dev), _rows(v, "v", dev, k.dtype, total, D)
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
            out_q, qo_rs = _new(q), Hq * D
        else:
            qo_rs = _rows(out_q, "out_q", dev, k.dtype, total, D)
            if out_q.shape != q.shape:
                raise ValueError("out_q must have q's shape")
    elif out_q is not None:
        raise ValueError("out_q needs q")
    if positions is not None:
        if rotary is None:
            raise ValueError("positions need rotary")
        _check_rotary(rotary, dev)
        _check_positions(positions, rotary, dev, total)
    turns, dim, inter, ms, axes, pair_axes = 0, 0, False, 1.0, 1, None
    if rotary is not None:
        _check_rotary(rotary, dev)
        turns, dim, inter, ms = _ptr(rotary.turns), rotary.dim, rotary.interleaved, rotary.attention_factor
        axes, pair_axes = rotary.num_axes, rotary.pair_axes
    if total == 0 or S == 0:
        return out_q
    rows = (_ptr(q), k.data_ptr(), v.data_ptr(), _DT[k.dtype], _ptr(cu_seqlens), kv_lengths.data_ptr(), page_table.data_ptr(), S,
            total, max_seqlen, Hq, Hk, D, q_rs, k_rs, v_rs, qo_rs, _ptr(positions))
    with _on(dev):
        if isinstance(cache, PagedKVCache4):
            abi.tri_attn_kv_append4(*rows, axes, _ptr(pair_axes), turns, dim, inter, ms, cache._c, MP, _ptr(out_q),
                                    _stream(dev))
            return out_q
        rest = (turns, dim, inter, ms, _ptr(cache.k), _ptr(cache.v), cache._code, _ptr(cache.k_scale),
                _ptr(cache.v_scale), cache.num_pages, cache.page_size, MP, cache._strides[0], cache._strides[1],
                _ptr(out_q), _stream(dev))
        if pair_axes is None:
            abi.tri_attn_kv_append(*rows, *rest)
        else:
            abi.tri_attn_kv_append_axes(*rows, axes, _ptr(pair_axes), *rest)
    return out_q


def kv_cache_read(cache: Union[PagedKVCache, PagedKVCache4], page_table, kv_lengths, cu_seqlens=None, max_seqlen=1,
                  total=None, *, dtype=None, out_k=None, out_v=None):
    """Rows of the cache back as packed (k, v), each (total, Hk, D).

    cu_seqlens (S + 1,) int32 splits the rows over the sequences (at most max_seqlen each; none is fine); without it
    there is one row for each sequence.  A sequence's rows are the last of its kv_lengths (S,) int32 slots, which may
    count fewer than it holds: a prefix for ``prompt_attention``, say.  total: rows of the outputs (at least the last
    entry of cu_seqlens; rows past that are left alone).  dtype: of the outputs where the cache holds codes (bfloat16
    by default), each rounded once.  out_k, out_v: outputs given, row-strided views among them.
    """
    if not isinstance(cache, _CACHES):
        raise TypeError("cache must be a PagedKVCache or a PagedKVCache4")
    cache._now()
    dev, Hk, D = cache.device, cache.heads, cache.head_dim
    if not cache.k.is_cuda:
        raise ValueError("kv_cache_read runs on CUDA tensors only")
    S, MP = _table(page_table, kv_lengths, cu_seqlens, dev)
    max_seqlen = int(max_seqlen)
    if total is None:
        if cu_seqlens is not None and out_k is None:
            raise ValueError("with cu_seqlens the rows of the outputs are counted by total, or by out_k")
        total = S if cu_seqlens is None else out_k.shape[0]
    total = int(total)
    if total < 0:
        raise ValueError("total must not be negative")
    if cu_seqlens is None and (total != S or max_seqlen != 1):
        raise ValueError("without cu_seqlens there is one row for each sequence")
    if (out_k is None) != (out_v is None):
        raise ValueError("out_k and out_v are given together")
    codes = isinstance(cache, PagedKVCache4) or cache.dtype == torch.float8_e4m3fn
    if dtype is None:
        dtype = out_k.dtype if out_k is not None else torch.bfloat16 if codes else cache.dtype
    if dtype not in _DT:
        raise TypeError("dtype must be float32, float16 or bfloat16")
    if not codes and dtype != cache.dtype:
        raise TypeError(f"the cache holds {cache.dtype}, and its rows come back as that")
    if out_k is None:
        out_k = torch.empty(total, Hk, D, dtype=dtype, device=dev)
        out_v = torch.empty_like(out_k)
        k_rs = v_rs = 0
    else:
        k_rs, v_rs = _rows(out_k, "out_k", dev, dtype, total, D), _rows(out_v, "out_v", dev, dtype, total, D)
        if out_k.shape[1] != Hk or out_v.shape[1] != Hk:
            raise ValueError(f"out_k and out_v must have the cache's {Hk} heads")
    if total == 0 or S == 0:
        return out_k, out_v
    seqs = (_ptr(cu_seqlens), _ptr(kv_lengths), _ptr(page_table), S, total, min(max_seqlen, total), Hk, D)
    outs = (_ptr(out_k), _ptr(out_v), _DT[dtype], k_rs, v_rs, _stream(dev))
    with _on(dev):
        if isinstance(cache, PagedKVCache4):
            abi.tri_attn_kv_read4(*seqs, cache._c, MP, *outs)
        else:
            abi.tri_attn_kv_read(*seqs, _ptr(cache.k), _ptr(cache.v), cache._code, _ptr(cache.k_scale),
                                 _ptr(cache.v_scale), cache.num_pages, cache.page_size, MP, cache._strides[0],
                                 cache._strides[1], *outs)
    return out_k, out_v


def paged_attention(q, cache: Union[PagedKVCache, PagedKVCache4], page_table, kv_lengths, cu_seqlens_q=None, max_seqlen_q=1, scale=None, *,
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
    of a key head).  A whole prompt, or a chunk of one with its prefix read back by ``kv_cache_read``, runs
    faster through ``prompt_attention``.
    """
    if not isinstance(cache, _CACHES):
        raise TypeError("cache must be a PagedKVCache or a PagedKVCache4")
    cache._now()
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    if q.dim() != 3:
        raise ValueError("expected q (total_q, Hq, D)")
    dev = q.device
    if not q.is_cuda:
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
        out = _new(q)
    else:
        _check_out(out, q.shape, q.dtype)
        _need(out, "out", dev)
    lse = torch.empty(Hq, total, dtype=torch.float32, device=dev) if return_aux else None
    if total and S:
        code = _DT[q.dtype]
        nbytes = abi.tri_attn_paged_workspace_size(code, max_seqlen_q, Hq, Hk, D)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        rows = (_ptr(q), code, _ptr(cu_seqlens_q), _ptr(kv_lengths), _ptr(page_table), S, total, max_seqlen_q, Hq, Hk, D,
                q_rs, s, 0 if window is None else _int32(window), _int32(sinks))
        outs = (_ptr(out), _ptr(lse), _ptr(ws), nbytes, _stream(dev))
        with _on(dev):
            if isinstance(cache, PagedKVCache4):
                abi.tri_attn_paged4_fwd(*rows, cache._c, MP, *outs)
            else:
                abi.tri_attn_paged_fwd(*rows, _ptr(cache.k), _ptr(cache.v), cache._code, _ptr(cache.k_scale),
                                       _ptr(cache.v_scale), cache.num_pages, cache.page_size, MP, cache._strides[0],
                                       cache._strides[1], *outs)
    return (out, lse) if return_aux else out
