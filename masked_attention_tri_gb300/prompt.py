"""Causal attention of whole prompts, or chunks of them, with grouped heads: forward, gradients, autograd.

Packed rows as in ``varlen_attention``, with as many query heads to a key head as the
model has; the work runs in libtriattn.so's kernels.
"""
from __future__ import annotations

import math

import torch

from . import abi
from .api import _DT, _check_out, _dense, _need, _new, _on, _ptr, _row_stride, _stream


def _prompt_args(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, scale):
    """The checked arguments that the forward and the backward share, in the C call's order."""
    for t, nm in ((q, "q"), (k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{nm} must be a torch.Tensor")
        if t.dim() != 3:
            raise ValueError("expected q (total_q, Hq, D) and k, v (total_k, Hk, D)")
    if not q.is_cuda:
        raise ValueError("prompt_attention runs on CUDA tensors only")
    dev, dtype, kv_shape = q.device, q.dtype, k.shape
    if dtype not in _DT:
        raise TypeError("q must be float32, float16 or bfloat16")
    if k.dtype != dtype or v.dtype != dtype:
        raise TypeError("q, k and v must share one dtype")
    total_q, Hq, D = q.shape
    total_k, Hk, Dk = kv_shape
    if Dk != D or v.shape != kv_shape:
        raise ValueError("k and v must share their shape and q's D")
    if Hk == 0 or Hq == 0 or Hq % Hk:
        raise ValueError(f"q's heads must be a multiple of k's {Hk}")
    strides = _row_stride(q, "q", dev), _row_stride(k, "k", dev), _row_stride(v, "v", dev)
    _need(cu_seqlens_q, "cu_seqlens_q", dev)
    _need(cu_seqlens_k, "cu_seqlens_k", dev)
    S = cu_seqlens_q.numel() - 1
    if (cu_seqlens_q.dtype != torch.int32 or cu_seqlens_k.dtype != torch.int32 or S < 0 or cu_seqlens_q.dim() != 1
            or cu_seqlens_k.dim() != 1 or cu_seqlens_k.numel() != S + 1):
        raise ValueError("cu_seqlens_q and cu_seqlens_k must be int32 with num_seqs + 1 entries each")
    if total_k == 0:  # (no key at all: some memory stands for the rows that no sequence has)
        k = v = torch.empty(1, Hk, D, dtype=dtype, device=dev)
        strides = strides[0], 0, 0
    s = 1.0 / math.sqrt(D) if scale is None else float(scale)
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), _DT[dtype], cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), S, total_q,
            total_k or 1, min(int(max_seqlen_q), total_q), min(int(max_seqlen_k), total_k), Hq, Hk, D, s, *strides)
    return args, S, (k, v)


def prompt_attention(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, scale=None, *, return_aux=False,
                     out=None):
    """Causal attention of packed prompts with grouped heads.

    q (total_q, Hq, D), k and v (total_k, Hk, D) with Hq a multiple of Hk (consecutive query heads share one);
    row-strided views are read in place.  cu_seqlens_q / cu_seqlens_k (S + 1,) int32 split the rows (at most
    max_seqlen_q / max_seqlen_k each; none is fine).  A sequence's queries are its newest tokens: of Lq queries and Lk
    keys, query j sees the keys up to Lk - Lq + j.  Equal lengths are whole prompts; more keys, chunks of prompts whose
    prefix is at hand (``kv_cache_read``).  scale defaults to 1/sqrt(D).  Returns O, or (O, lse) with return_aux (lse
    float32 (Hq, total_q)); a query that sees no key gets O = 0 and lse = -inf; rows past the last entry of
    cu_seqlens_q are left alone.
    """
    args, S, hold = _prompt_args(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, scale)
    dev = q.device
    if out is None:
        out = _new(q)
    else:
        _check_out(out, q.shape, q.dtype)
        _need(out, "out", dev)
    lse = torch.empty(q.shape[1], q.shape[0], dtype=torch.float32, device=dev) if return_aux else None
    if q.shape[0] and S:
        with _on(dev):
            abi.tri_attn_prompt_fwd(*args, _ptr(out), _ptr(lse), _stream(dev))
    return (out, lse) if return_aux else out


def prompt_attention_backward(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, out, lse, d_out,
                              scale=None):
    """(dq, dk, dv) of ``prompt_attention`` from its inputs, its O and lse, and dL/dO.

    dk and dv are summed over the query heads that share a key head.  Rows past the last entries of cu_seqlens_q and
    cu_seqlens_k are not written.
    """
    args, S, hold = _prompt_args(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, scale)
    dev, (total_q, Hq, D) = q.device, q.shape
    for t, nm in ((out, "out"), (d_out, "d_out")):
        _need(t, nm, dev)
        if t.shape != q.shape or t.dtype != q.dtype:
            raise ValueError(f"{nm} must have q's shape and dtype")
    _need(lse, "lse", dev)
    if lse.dtype != torch.float32 or tuple(lse.shape) != (Hq, total_q):
        raise ValueError(f"lse must be float32 {(Hq, total_q)}")
    dq, dk, dv = _new(q), _new(k), _new(k)
    if total_q == 0:  # (keys that no query sees)
        return dq, dk.zero_(), dv.zero_()
    if S:
        nbytes = abi.tri_attn_prompt_bwd_workspace_size(*args[3:4], *args[6:14])
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        gk, gv = (dk, dv) if k.shape[0] else hold
        with _on(dev):
            abi.tri_attn_prompt_bwd(*args, _ptr(lse), _ptr(out), _ptr(d_out), _ptr(dq), _ptr(gk), _ptr(gv), _ptr(ws),
                                    nbytes, _stream(dev))
    return dq, dk, dv


def _zero_rest(x, cu):
    """Zeros into the rows of x that no sequence of cu has (what comes after sums over all rows)."""
    total, H, D = x.shape
    if total:
        with _on(x.device):
            abi.tri_attn_zero_rest(_ptr(x), _DT[x.dtype], _ptr(cu), cu.numel() - 1, total, H, D, _stream(x.device))
    return x


class _PromptFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_q, cu_k, max_q, max_k, scale):
        out, lse = prompt_attention(q, k, v, cu_q, cu_k, max_q, max_k, scale, return_aux=True)
        _zero_rest(out, cu_q)
        ctx.save_for_backward(q, k, v, cu_q, cu_k, out, lse)
        ctx.sizes = max_q, max_k, scale
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_out):
        q, k, v, cu_q, cu_k, out, lse = ctx.saved_tensors
        max_q, max_k, scale = ctx.sizes
        dq, dk, dv = prompt_attention_backward(q, k, v, cu_q, cu_k, max_q, max_k, out, lse, _dense(d_out), scale)
        return _zero_rest(dq, cu_q), _zero_rest(dk, cu_k), _zero_rest(dv, cu_k), None, None, None, None, None


def prompt_attention_autograd(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, scale=None):
    """``prompt_attention`` (O alone) with gradients for q, k and v (of first order).

    Rows that belong to no sequence (before the first entries of cu_seqlens and from the last ones on) get O = 0 and
    gradients of 0, whatever they hold.

    Its backward may be captured into a graph, as any autograd function's, only while no
    graph of the same leaves made outside the capture lives (PyTorch ties the leaves'
    accumulation to the stream of the first).
    """
    return _PromptFn.apply(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, scale)
