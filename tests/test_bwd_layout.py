"""Shared memory of the tensor-core backward: how long a packed sequence may be, and gradients on both sides of the
length where the rows' lse leave it.

The host program below runs the library's own arithmetic (csrc/bwd_layout.h).
"""
import math
import os
import shutil
import subprocess

import pytest
import torch

from masked_attention_tri_gb300 import build

PROGRAM = r"""
#include <cstdio>
#include "bwd_layout.h"
using namespace triattn::tc;
int main() {
    int D, bias, max_q, two;
    while (std::scanf("%d %d %d %d", &D, &bias, &max_q, &two) == 4) {
        BwdShape s;
        const bool ok = bwd_shape(s, D, bias, max_q, two != 0);
        std::printf("%d %d %d %d %u\n", ok, ok ? s.qs : 0, ok ? s.lse_row : 0, ok ? s.lo : 0,
                    ok ? bwd_layout(s, (D + 63) / 64).total + kBwdAlign : 0u);
    }
}
"""


@pytest.fixture(scope="module")
def shape(tmp_path_factory):
    d = tmp_path_factory.mktemp("layout")
    src, exe = d / "layout.cpp", d / "layout"
    src.write_text(PROGRAM)
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", build.CSRC, str(src), "-o", str(exe)], check=True)

    def run(*a):
        r = subprocess.run([str(exe)], input=" ".join(str(x) for x in a), capture_output=True, text=True, check=True)
        ok, qs, row, lo, total = (int(x) for x in r.stdout.split())
        assert total <= 227 * 1024
        return (qs, row, lo) if ok else None
    return run


def _limit(D, bias):
    """The longest packed sequence: beside the fixed parts (K, V, one stage of Q and dO, dS, the bias, dQ's staging, two
    rows of 128 sums, 20 barriers and three words, 1 KB of alignment) 4 bytes for each 128 queries, in steps of 16 bytes."""
    box = 16384 * (2 if D > 64 else 1)
    shared = 4 if D > 64 and bias == 4 else bias  # (an fp32 bias with D > 64: one half at a time)
    b = 0 if not bias else (32768 if shared == 2 or D > 64 else 65536)
    left = 227 * 1024 - 1024 - (4 * box + 2 * 16384 + b + 32768 + 2 * 512 + 160 + 12)
    return left // 16 * 4 * 128


@pytest.mark.parametrize("D", [64, 80, 128])
@pytest.mark.parametrize("bias", [0, 2, 4])
def test_longest_sequence(shape, D, bias):
    n = _limit(D, bias)
    assert shape(D, bias, n, 0) is not None and shape(D, bias, n + 1, 0) is None
    if D > 64 and bias:
        assert n == 27136


def test_where_the_lse_row_leaves(shape):
    assert shape(128, 2, 10752, 0) == (1, 1, 0) and shape(128, 2, 10753, 0) == (1, 0, 0)
    assert shape(128, 4, 100, 0) == (1, 0, 0)
    assert shape(64, 2, 2048, 0) == (2, 1, 0)
    # dS in two pieces: always with D <= 64 at these lengths, up to 84 q blocks above
    assert shape(64, 0, 100000, 1) == (2, 1, 1)
    assert shape(128, 0, 84 * 128, 1) == (1, 1, 1) and shape(128, 0, 84 * 128 + 1, 1) == (1, 1, 0)
    # the triangle form
    assert shape(64, 2, -1, 0) == (2, 1, 0) and shape(64, 4, -1, 0) == (1, 1, 0)
    assert shape(128, 2, -1, 0) == (1, 1, 0) and shape(128, 4, -1, 0) == (1, 0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("L", [10752, 10753, 27136, 27137])
@pytest.mark.parametrize("mask", ["causal", "prefix_lm"])
def test_gradients_with_a_bias_of_long_sequences(L, mask):
    """16-bit bias, heads of 128, more queries than keys (so that the bias stays small).  Tolerances as in
    test_sink_window.py's test_gradients_with_a_bias."""
    import masked_attention_tri_gb300 as ta
    D, Lk, u, s = 128, 136, 2.0 ** -8, 1 / math.sqrt(128)
    g = torch.Generator().manual_seed(L)
    q, d_out = (torch.randn(L, 1, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    k, v = (torch.randn(Lk, 1, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    bias = torch.randn(1, L, Lk, generator=g).to(torch.bfloat16).cuda()
    cq, ck = (torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (L, Lk))
    kw = dict(mask_mod=mask, bias=bias, **(dict(prefix_lengths=70) if mask == "prefix_lm" else {}))
    o, lse, _ = ta.varlen_attention(q, k, v, cq, ck, L, Lk, return_aux=True, **kw)
    got = ta.varlen_attention_backward(q, k, v, cq, ck, L, Lk, o, lse, d_out, **kw)
    torch.cuda.synchronize()
    assert ta.get_status() == 0
    Q, K, V, G, B = (x.double() for x in (q[:, 0], k[:, 0], v[:, 0], d_out[:, 0], bias[0]))
    i, j = torch.arange(L, device="cuda")[:, None], torch.arange(Lk, device="cuda")
    keep = (j <= i) if mask == "causal" else (j <= i) | (j < 70)
    P = (s * Q @ K.t() + B).masked_fill(~keep, -math.inf).softmax(-1)
    O, dP = P @ V, G @ V.t()
    delta = (G * O).sum(-1, keepdim=True)
    dS = P * (dP - delta)
    tO = 2 * u * (P @ V.abs())
    m = P * ((u + u / 8) * (dP.abs() + delta.abs()) + (G.abs() * tO).sum(-1, keepdim=True))
    want = (s * dS @ K, s * dS.t() @ Q, P.t() @ G, dS)
    tols = (s * m @ K.abs(), s * m.t() @ Q.abs(), (u + u / 8) * P.t() @ G.abs(), m)
    for name, x, y, tol in zip(("dq", "dk", "dv", "dbias"), got, want, tols):
        err = (x.double().reshape(y.shape) - y).abs()
        assert bool((err <= tol + u * y.abs()).all()), (name, float((err - tol - u * y.abs()).max()))
