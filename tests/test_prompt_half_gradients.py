"""fp16 gradients of prompt attention for dO far from 1: a mean loss' (1e-4 and less), large ones, rows of unlike sizes.

Tolerances.  On tensor cores P and dS are operands of 16 bits, held times powers of two: P, at most 1, times 2^14, off by
eps / 2 |P| or half of fp16's least step, 2^-25 2^-14; dS times 2^e with B 2^e in [2^14, 2^15), B the bound |dO| max |V| + |delta| of
the row (dQ) or the largest of the sequence's rows of a key head (dK), so 2^-e <= 2^-14 B: off by eps / 2 |dS| (one number; no
more as two) or 2^-25 2^-14 B, with a hundredth for the bound's own fp32 sums.  The rest is fp32's: `reference` of the same numbers held in fp32, twice,
as the kernel's sums run in another order.  The result is off by eps / 2 of itself, or 2^-25.
"""
import math

import pytest
import torch

from masked_attention_tri_gb300 import abi, build
from test_prompt_attention import F16, _cu, _i32, _inputs, reference


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def test_workspace():
    """fp16 on tensor cores: |dO| of the rows and three numbers a (sequence, key head) beside delta."""
    size = abi.tri_attn_prompt_bwd_workspace_size
    assert size(abi.TA_F16, 1, 100, 100, 100, 100, 4, 2, 64) == (448 + 448 + 64) * 4
    assert size(abi.TA_F16, 40, 100, 100, 100, 100, 4, 2, 64) == (448 + 448 + 256) * 4
    assert size(abi.TA_F16, 1, 100, 100, 100, 100, 4, 2, 256) == 448 * 4
    assert size(abi.TA_F16, 1, 1000, 1000, 1000, 1000, 4, 2, 64) == (2 * 4032 + 64 + 4 * 2 * 1000 * 2 * 64) * 4


def _check(q, k, v, g, lq, lk):
    """Checks all gradients; returns the kernel's and the exact ones."""
    import masked_attention_tri_gb300 as ta
    Hq, Hk, D = q.shape[1], k.shape[1], q.shape[2]
    cu_q, cu_k, s = _i32(_cu(lq)), _i32(_cu(lk)), float(torch.tensor(1 / math.sqrt(D), dtype=torch.float32))
    o, lse = ta.prompt_attention(q, k, v, cu_q, cu_k, max(lq), max(lk), return_aux=True)
    got = dict(zip(("dq", "dk", "dv"), ta.prompt_attention_backward(q, k, v, cu_q, cu_k, max(lq), max(lk), o, lse, g)))
    R, T = reference(q.float(), k.float(), v.float(), lq, lk, s, g.float(), out=o.float())
    eps, G = torch.finfo(F16).eps, Hq // Hk
    piece = {n: torch.zeros_like(R[n]) for n in got}
    for a, b, c, d in zip(_cu(lq), _cu(lq)[1:], _cu(lk), _cu(lk)[1:]):
        if a == b or c == d:
            continue
        n, m = b - a, d - c
        hide = torch.arange(m, device="cuda") > torch.arange(m - n, m, device="cuda")[:, None]
        for hk in range(Hk):
            K, V = k[c:d, hk].double(), v[c:d, hk].double()
            heads = range(hk * G, hk * G + G)
            delta = {h: (g[a:b, h].double() * o[a:b, h].double()).sum(1) for h in heads}
            size = {h: g[a:b, h].double().norm(dim=1) for h in heads}
            far = V.norm(dim=1).max()
            all_rows = far * max(float(x.max()) for x in size.values()) + max(float(x.abs().max()) for x in delta.values())
            for h in heads:
                Q, dO = q[a:b, h].double(), g[a:b, h].double()
                P = (s * (Q @ K.t())).masked_fill(hide, -math.inf).softmax(1).nan_to_num(0.0)
                dS = P * (dO @ V.t() - delta[h][:, None])
                seen = (~hide).double()
                step = 1.01 * 2.0 ** -39 * (far * size[h] + delta[h].abs())[:, None]
                piece["dq"][a:b, h] += s * (dS.abs() * eps / 2 + step * seen) @ K.abs()
                piece["dk"][c:d, hk] += s * (dS.abs() * eps / 2 + 1.01 * 2.0 ** -39 * all_rows * seen).t() @ Q.abs()
                piece["dv"][c:d, hk] += (P * eps / 2 + 2.0 ** -39 * seen).t() @ dO.abs()
    for name, x in got.items():
        tol = (eps / 2 * R[name].abs()).clamp_min(2.0 ** -25) + 2 * (T[name] + piece[name])
        off = (x.double() - R[name]).abs() - tol
        # (a result of 65520 or more, half a step past fp16's largest number 65504, is an infinity when it is rounded to nearest)
        off[torch.isinf(x) & (x.sign() == R[name].sign()) & (R[name].abs() + tol >= 65520)] = 0
        assert bool((off <= 0).all()), (name, int((off > 0).sum()), float(off.max()))
    assert ta.get_status() == 0
    return got, R


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("lq,lk", [([4096], [4096]), ([700, 130], [5000, 130])])
@pytest.mark.parametrize("up", [6, -6])
def test_small_dO(lq, lk, D, up):
    """dO about 2^-14 and thousands of keys; keys times 2^up and queries by it, so that dQ (or dK) itself is no subnormal."""
    q, k, v, g = _inputs(lq, lk, 4, 2, D, F16)
    got, R = _check((q * 2.0 ** -up).to(F16), (k * 2.0 ** up).to(F16), v, (g * 2.0 ** -14).to(F16), lq, lk)
    name = "dq" if up > 0 else "dk"
    off, size = (got[name].double() - R[name]).norm(), R[name].norm()
    assert float(size) > 0 and float(off / size) < 0.02


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_large_dO(D):
    """dO V past what fp16 holds: dS is a number all the same, where keys are small dQ, and where queries are dK."""
    lq, lk = [200, 40], [300, 40]
    q, k, v, g = _inputs(lq, lk, 4, 2, D, F16)
    got, _ = _check(q, (k * 2.0 ** -7).to(F16), v * 32, g * 1000, lq, lk)
    assert bool(torch.isfinite(got["dq"]).all())
    got, _ = _check((q * 2.0 ** -9).to(F16), k, v * 32, g * 1000, lq, lk)
    assert bool(torch.isfinite(got["dk"]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_rows_of_unlike_sizes(D):
    """Each row of dQ keeps its own precision; sequences and rows 2^-12 and 2^-20 of others, and rows and sequences of zeros."""
    lq, lk = [600, 520, 100, 30], [900, 520, 100, 30]
    q, k, v, g = _inputs(lq, lk, 6, 2, D, F16)
    by = torch.ones(sum(lq), 1, 1, device="cuda")
    by[100:200] = 2.0 ** -12
    by[300:310] = 0
    by[600:1120] = 2.0 ** -12
    by[1120:1220] = 0
    by[1220:] = 2.0 ** -20
    got, _ = _check(q, k, v, (g * by).to(F16), lq, lk)
    assert bool((got["dq"][1120:1220] == 0).all()) and bool((got["dv"][1420:1520] == 0).all())


@pytest.mark.gpu
def test_infinities_stay_in_their_sequence():
    """NaN and infinities of one sequence change nothing in another's gradients."""
    import masked_attention_tri_gb300 as ta
    lq = [200, 70, 130]
    q, k, v, g = _inputs(lq, lq, 4, 2, 64, F16)
    cu = _i32(_cu(lq))
    o, lse = ta.prompt_attention(q, k, v, cu, cu, 200, 200, return_aux=True)
    want = ta.prompt_attention_backward(q, k, v, cu, cu, 200, 200, o, lse, g)
    v2, g2 = v.clone(), g.clone()
    v2[210], g2[220], g2[230] = math.inf, math.nan, math.inf
    o, lse = ta.prompt_attention(q, k, v2, cu, cu, 200, 200, return_aux=True)
    got = ta.prompt_attention_backward(q, k, v2, cu, cu, 200, 200, o, lse, g2)
    for a, b in zip(want, got):
        assert torch.equal(a[:200], b[:200]) and torch.equal(a[270:], b[270:])
        assert not bool(torch.isfinite(b[200:270]).all())
