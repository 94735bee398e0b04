"""prompt_attention_autograd of packed buffers that are longer than their sequences, and gradients that come as views.

Rows that no sequence has get O = 0 and gradients of exactly 0, whatever the inputs, dO or freshly allocated memory hold there:
a projection's weight gradient sums over all rows.
"""
import math

import pytest
import torch

from masked_attention_tri_gb300 import abi, build
from test_prompt_attention import A, BF, F16, F32, _cu, _i32, _inputs


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _zero(**kw):
    args = dict(x=A, dtype=abi.TA_BF16, cu_seqlens=A, num_seqs=2, total=8, H=2, D=64, stream=0)
    args.update(kw)
    return abi.tri_attn_zero_rest(**args)


@pytest.mark.parametrize("kw,exc", [(dict(x=0), ValueError), (dict(cu_seqlens=0), ValueError), (dict(num_seqs=-1), ValueError),
                                    (dict(total=-1), ValueError), (dict(H=0), ValueError), (dict(D=0), ValueError),
                                    (dict(x=A + 8), ValueError), (dict(cu_seqlens=A + 2), ValueError),
                                    (dict(dtype=abi.TA_E4M3), ValueError), (dict(D=4), NotImplementedError),
                                    (dict(D=264), NotImplementedError)])
def test_zero_rest_refuses(kw, exc):
    with pytest.raises(exc):
        _zero(**kw)


def test_zero_rest_of_nothing():
    _zero(total=0)


def _fill_nan(*like):
    """What the allocator hands out next holds NaN."""
    for _ in range(2):
        held = [torch.full(t.shape, math.nan, dtype=t.dtype, device="cuda") for t in like for _ in range(4)]
        del held
    torch.cuda.synchronize()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF, 128), (F16, 64), (F32, 64), (BF, 200), (F32, 4)])
@pytest.mark.parametrize("before,behind", [(0, 0), (0, 1), (0, 130), (5, 0), (3, 300)])
def test_rows_of_no_sequence(dtype, D, before, behind):
    import masked_attention_tri_gb300 as ta
    lq, lk, Hq, Hk = [70, 0, 200], [90, 4, 200], 4, 2
    q, k, v, g = _inputs(lq, lk, Hq, Hk, D, dtype, extra=before + behind)
    nq, nk = sum(lq), sum(lk)
    for t, n in ((q, nq), (k, nk), (v, nk), (g, nq)):
        t[:before] = math.nan
        t[before + n:] = math.nan
    cu_q, cu_k = _i32([before + x for x in _cu(lq)]), _i32([before + x for x in _cu(lk)])
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    _fill_nan(q, k)
    o = ta.prompt_attention_autograd(*leaves, cu_q, cu_k, 200, 200)
    _fill_nan(q, k)
    got = torch.autograd.grad(o, leaves, g)
    want, lse = ta.prompt_attention(q, k, v, cu_q, cu_k, 200, 200, return_aux=True)
    d = ta.prompt_attention_backward(q, k, v, cu_q, cu_k, 200, 200, want, lse, g)
    for x, w, n in ((o, want, nq), (got[0], d[0], nq), (got[1], d[1], nk), (got[2], d[2], nk)):
        assert torch.equal(x[before:before + n], w[before:before + n])
        assert bool((x[:before] == 0).all()) and bool((x[before + n:] == 0).all())
    assert ta.get_status() == 0


@pytest.mark.gpu
def test_no_sequence_at_all():
    import masked_attention_tri_gb300 as ta
    q, k, v, g = _inputs([30], [40], 4, 2, 64, BF)
    leaves = [t.requires_grad_() for t in (q, k, v)]
    _fill_nan(q, k)
    o = ta.prompt_attention_autograd(*leaves, _i32([0]), _i32([0]), 0, 0)
    _fill_nan(q, k)
    assert bool((o == 0).all()) and all(bool((x == 0).all()) for x in torch.autograd.grad(o, leaves, g))


@pytest.mark.gpu
def test_rows_of_no_sequence_captured():
    """The offsets are read on the device: a replayed graph zeroes the rows that are left over then."""
    import masked_attention_tri_gb300 as ta
    q, k, v, g = _inputs([300], [300], 4, 2, 64, BF)
    cu = _i32([0, 100, 250])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        leaves = [t.detach().requires_grad_() for t in (q, k, v)]
        o = ta.prompt_attention_autograd(*leaves, cu, cu, 300, 300)
        d = torch.autograd.grad(o, leaves, g)
    for ends in ([0, 100, 250], [0, 200, 300], [20, 30, 40]):
        cu.copy_(_i32(ends))
        for x in (o, *d):
            x.detach().fill_(math.nan)
        graph.replay()
        for x in (o, *d):
            a, b = ends[0], ends[-1]
            assert bool((x[:a] == 0).all()) and bool((x[b:] == 0).all()) and bool(torch.isfinite(x[a:b]).all())
    assert ta.get_status() == 0
