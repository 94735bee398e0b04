"""Rotary positions of packed queries and keys, forward and backward.

The layout is the packed form's: (total, H, D) rows of several sequences, one
int32 position for each row.  The work runs in libtriattn.so's kernels.
"""
from __future__ import annotations

import math
from typing import Optional

import torch

from . import abi
from .api import _DT, _dense, _need, _new, _on, _ptr, _row_stride, _stream

_SCALINGS = (None, "linear", "ntk", "yarn")


def _pair_axes(sections, pairs, layout):
    """The axis of each pair."""
    want = [int(n) for n in sections]
    if not want or min(want) < 1 or sum(want) != pairs:
        raise ValueError(f"sections must be positive and add up to dim / 2 = {pairs}")
    if layout == "blocks":
        return [a for a, n in enumerate(want) for _ in range(n)]
    if layout != "interleaved":
        raise ValueError("section_layout must be 'blocks' or 'interleaved'")
    axes = []
    while len(axes) < pairs:
        for a in range(len(want)):
            if want[a]:
                want[a] -= 1
                axes.append(a)
    return axes


class Rotary:
    """The frequencies of rotary positions, kept on one device for any number of calls.

    dim: the leading elements of a head that turn (even).  Pair i turns by
    position * theta_i, theta_i = base^(-2i / dim); interleaved pairs elements
    (2i, 2i + 1), otherwise (i, i + dim / 2).  scaling, for contexts beyond
    ``original_length`` positions by ``factor``:

    * None: as above;
    * "linear": theta_i / factor (position interpolation);
    * "ntk": base * factor^(dim / (dim - 2)) in place of base;
    * "yarn": by parts (Peng et al., "YaRN", section 3.2): with r_i = original_length
      theta_i / 2 pi turns in the original context, theta_i is kept where r_i >=
      beta_fast, divided by factor where r_i <= beta_slow and blended linearly in
      r_i between; cos and sin are multiplied by 0.1 ln(factor) + 1.

    attention_factor replaces that multiplier (1 without "yarn").

    sections: pairs of each axis where a token has a position on several (time, height, width;
    their sum is dim / 2).  Calls then take positions (axes, total), and pair i turns by
    its axis' position.  section_layout "blocks": the first sections[0] pairs are axis 0's, the
    next axis 1's, and so on; "interleaved": the pairs go round the axes that still want
    some (0, 1, 2, 0, 1, 2, ...).  section_frequencies "shared": theta_i as above, over all pairs;
    "own": over the axis' own pairs (theta = base^(-j / sections[a]) for its j-th; without scaling).
    """

    def __init__(self, dim, base=10000.0, *, interleaved=False, scaling=None, factor=1.0, original_length=0,
                 beta_fast=32.0, beta_slow=1.0, attention_factor=None, sections=None, section_layout="blocks",
                 section_frequencies="shared", device=None):
        dim, factor = int(dim), float(factor)
        if dim < 2 or dim % 2:
            raise ValueError("dim must be even and at least 2")
        if scaling not in _SCALINGS:
            raise ValueError(f"scaling must be one of {[s for s in _SCALINGS if s]} or None")
        if not base > 0 or not factor >= 1 or math.isinf(base) or math.isinf(factor):
            raise ValueError("base must be positive and factor at least 1")
        if scaling is None and factor != 1.0:
            raise ValueError("factor needs a scaling")
        if scaling == "ntk":
            if dim < 4:
                raise ValueError("ntk scaling needs dim >= 4")
            base = base * factor ** (dim / (dim - 2))
        axes = None if sections is None else _pair_axes(sections, dim // 2, section_layout)
        if section_frequencies not in ("shared", "own"):
            raise ValueError("section_frequencies must be 'shared' or 'own'")
        theta = [base ** (-2.0 * i / dim) for i in range(dim // 2)]
        if section_frequencies == "own":
            if sections is None or scaling is not None:
                raise ValueError("frequencies of each section's own need sections and no scaling")
            place = [axes[:i].count(a) for i, a in enumerate(axes)]
            theta = [base ** (-float(j) / int(sections[a])) for a, j in zip(axes, place)]
        if scaling == "linear":
            theta = [t / factor for t in theta]
        if scaling == "yarn":
            if original_length <= 0 or not beta_fast > beta_slow:
                raise ValueError("yarn scaling needs original_length > 0 and beta_fast > beta_slow")

            def blend(t):
                keep = (original_length * t / (2 * math.pi) - beta_slow) / (beta_fast - beta_slow)
                keep = min(1.0, max(0.0, keep))
                return keep * t + (1 - keep) * t / factor
            theta = [blend(t) for t in theta]
        if attention_factor is None:
            attention_factor = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0
        self.dim = dim
        self.interleaved = bool(interleaved)
        self.attention_factor = float(attention_factor)
        self.theta = theta
        # turns per position as 64-bit fixed point (two's complement in an int64 tensor)
        turns = [int(round(t / (2 * math.pi) * 2.0 ** 64)) & (2 ** 64 - 1) for t in theta]
        turns = [t - 2 ** 64 if t >= 2 ** 63 else t for t in turns]
        self.turns = torch.tensor(turns, dtype=torch.int64, device=device)
        self.num_axes = 1 if axes is None else len(sections)
        self.pair_axes = None if axes is None else torch.tensor(axes, dtype=torch.int32, device=self.turns.device)

    def positions_shape(self, total):
        """The shape of a call's positions."""
        return (total,) if self.pair_axes is None else (self.num_axes, total)

    @property
    def device(self) -> torch.device:
        return self.turns.device


def _rotary_rows(t, name, dev, dtype, total):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 3 or t.shape[0] != total:
        raise ValueError(f"{name} must be (total, H, D) with total = {total}")
    if t.dtype != dtype:
        raise TypeError("q and k must share one dtype")
    return _row_stride(t, name, dev)


def _check_rotary(rotary, dev):
    if not isinstance(rotary, Rotary):
        raise TypeError("rotary must be a Rotary")
    if rotary.turns.device != dev:
        raise ValueError(f"rotary is on {rotary.turns.device}, expected {dev}")


def _check_positions(positions, rotary, dev, total):
    _need(positions, "positions", dev)
    if rotary.pair_axes is None:
        if positions.dtype != torch.int32 or positions.numel() != total:
            raise ValueError("positions must be int32 with one entry per row")
    elif positions.dtype != torch.int32 or tuple(positions.shape) != (rotary.num_axes, total):
        raise ValueError(f"positions must be int32 (axes, rows) = {(rotary.num_axes, total)}")


def _rotary_call(q, k, positions, rotary, inverse, out_q, out_k):
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    if q.dim() != 3:
        raise ValueError("expected q (total, Hq, D)")
    dev = q.device
    if not q.is_cuda:
        raise ValueError("rotary_embedding runs on CUDA tensors only")
    if q.dtype not in _DT:
        raise TypeError("q must be float32, float16 or bfloat16")
    total, Hq, D = q.shape
    q_rs = _rotary_rows(q, "q", dev, q.dtype, total)
    _check_rotary(rotary, dev)
    _check_positions(positions, rotary, dev, total)
    Hk, k_rs, ko_rs = 0, 0, 0
    if k is None and out_k is not None:
        raise ValueError("out_k needs k")
    if k is not None:
        k_rs = _rotary_rows(k, "k", dev, q.dtype, total)
        Hk = k.shape[1]
        if k.shape[2] != D:
            raise ValueError("k must have q's D")
        if out_k is None:
            out_k, ko_rs = _new(k), Hk * D
        else:
            ko_rs = _rotary_rows(out_k, "out_k", dev, q.dtype, total)
            if out_k.shape != k.shape:
                raise ValueError("out_k must have k's shape")
    if out_q is None:
        out_q, qo_rs = _new(q), Hq * D
    else:
        qo_rs = _rotary_rows(out_q, "out_q", dev, q.dtype, total)
        if out_q.shape != q.shape:
            raise ValueError("out_q must have q's shape")
    if total:
        args = (_ptr(rotary.turns), rotary.dim, rotary.interleaved, rotary.attention_factor, inverse, total, Hq, Hk, D,
                q_rs, k_rs, qo_rs, ko_rs, _ptr(out_q), _ptr(out_k), _stream(dev))
        with _on(dev):
            if rotary.pair_axes is None:
                abi.tri_attn_rotary(_ptr(q), _ptr(k), _DT[q.dtype], _ptr(positions), *args)
            else:
                abi.tri_attn_rotary_axes(_ptr(q), _ptr(k), _DT[q.dtype], _ptr(positions), rotary.num_axes,
                                         _ptr(rotary.pair_axes), *args)
    return out_q if k is None else (out_q, out_k)


def rotary_embedding(q, k, positions, rotary: Rotary, *, out_q=None, out_k=None):
    """q (total, Hq, D) and k (total, Hk, D) turned by their rows' positions.

    positions: int32 (total,), any values; (axes, total) where rotary has sections.  k may be None (then q alone is
    returned, else (q, k)).  q, k and the outputs may be row-strided views (heads
    and elements contiguous), such as the slices of an interleaved QKV buffer;
    out_q=q / out_k=k turn in place.  fp32 arithmetic, one rounding.
    """
    return _rotary_call(q, k, positions, rotary, False, out_q, out_k)


def rotary_embedding_backward(d_q, d_k, positions, rotary: Rotary, *, out_q=None, out_k=None):
    """Gradients of ``rotary_embedding``: the turn by the opposite angle.  Arguments as there."""
    return _rotary_call(d_q, d_k, positions, rotary, True, out_q, out_k)


class _RotaryFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, rotary, inverse):
        ctx.save_for_backward(positions)
        ctx.rotary, ctx.inverse = rotary, inverse
        return _rotary_call(q, k, positions, rotary, inverse, None, None)

    @staticmethod
    def backward(ctx, d_q, d_k=None):
        # (the turn is linear: its gradient is the opposite turn, itself differentiable, for second derivatives)
        (positions,) = ctx.saved_tensors
        if d_k is None:
            return _RotaryFn.apply(_dense(d_q), None, positions, ctx.rotary, not ctx.inverse), None, None, None, None
        d_q, d_k = _RotaryFn.apply(_dense(d_q), _dense(d_k), positions, ctx.rotary, not ctx.inverse)
        return d_q, d_k, None, None, None


def rotary_embedding_autograd(q, k: Optional[torch.Tensor], positions, rotary: Rotary):
    """``rotary_embedding`` with gradients for q and k, of any order.

    Its backward may be captured into a graph, as any autograd function's, only while no
    graph of the same leaves made outside the capture lives (PyTorch ties the leaves'
    accumulation to the stream of the first).
    """
    return _RotaryFn.apply(q, k, positions, rotary, False)
