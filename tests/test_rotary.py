"""Rotary positions: refusals and frequencies on the CPU, values and gradients on the GPU.

The reference turns each pair in fp64 from the definition.  Tolerance, for a pair
(a, b) and a result y: half a step of the output type, eps / 2 |y|, plus the fp32
arithmetic's (|a| + |b|) m 2^-21: cos and sin off by 2^-23 (their function) and 2^-25 (their
argument), the factor m by 2^-24, two products and a sum by 3 * 2^-24.
"""
import math

import pytest
import torch

from masked_attention_tri_gb300 import abi, build

A = 0x10000


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _theta(dim, base=10000.0):
    return [base ** (-2.0 * i / dim) for i in range(dim // 2)]


def _turn64(x, positions, rotary, back=False):
    """fp64 definition; rotary.theta holds the radians per position."""
    th = torch.tensor(rotary.theta, dtype=torch.float64)
    ang = positions.double().cpu()[:, None] * th
    c, s = (ang.cos() * rotary.attention_factor)[:, None], (ang.sin() * rotary.attention_factor)[:, None]
    s = -s if back else s
    y, n = x.double().cpu().clone(), rotary.dim // 2
    i0, i1 = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if rotary.interleaved else (slice(0, n), slice(n, 2 * n))
    a, b = y[..., i0].clone(), y[..., i1].clone()
    mag = torch.zeros_like(y)
    mag[..., i0] = mag[..., i1] = a.abs() + b.abs()
    y[..., i0], y[..., i1] = a * c - b * s, a * s + b * c
    return y, mag * rotary.attention_factor


def _check(got, want, mag):
    err = (got.double().cpu() - want).abs()
    tol = torch.finfo(got.dtype).eps / 2 * want.abs() + mag * 2.0 ** -21
    assert bool((err <= tol).all()), float((err - tol).max())


# ---------------------------------------------------------------------------- CPU

def test_frequencies():
    import masked_attention_tri_gb300 as ta
    plain = ta.Rotary(64)
    assert plain.theta == _theta(64) and plain.attention_factor == 1.0
    assert ta.Rotary(64, scaling="linear", factor=4.0).theta == [t / 4 for t in _theta(64)]
    ntk = ta.Rotary(64, scaling="ntk", factor=4.0)
    assert ntk.theta == _theta(64, 10000.0 * 4.0 ** (64 / 62))
    assert abs(ntk.theta[-1] * 4.0 / _theta(64)[-1] - 1) < 1e-12  # the slowest pair is stretched by the factor
    y = ta.Rotary(64, scaling="yarn", factor=8.0, original_length=4096)
    for t, u in zip(_theta(64), y.theta):
        turns = 4096 * t / (2 * math.pi)
        if turns >= 32:
            assert u == t
        elif turns <= 1:
            assert abs(u * 8 / t - 1) < 1e-12
        else:
            assert t / 8 < u < t
    assert abs(y.attention_factor - (0.1 * math.log(8.0) + 1)) < 1e-15
    # the fixed point is a fraction of a turn
    for t, f in zip(plain.turns.tolist(), plain.theta):
        assert abs((t % 2 ** 64) / 2 ** 64 - f / (2 * math.pi)) < 2e-17


@pytest.mark.parametrize("kw", [dict(dim=7), dict(dim=0), dict(dim=8, scaling="other"), dict(dim=8, factor=2.0),
                                dict(dim=2, scaling="ntk", factor=2.0), dict(dim=8, scaling="linear", factor=0.5),
                                dict(dim=8, scaling="yarn", factor=2.0), dict(dim=8, base=0.0)])
def test_frequencies_refused(kw):
    import masked_attention_tri_gb300 as ta
    with pytest.raises(ValueError):
        ta.Rotary(**kw)


def _call(**kw):
    args = dict(q=A, k=A, dtype=abi.TA_BF16, positions=A, turns=A, rotary_dim=64, interleaved=0, mscale=1.0, inverse=0,
                total=4, Hq=4, Hk=2, D=64, q_row_stride=0, k_row_stride=0, q_out_row_stride=0, k_out_row_stride=0,
                q_out=A + 0x10000, k_out=A + 0x20000, stream=0)
    args.update(kw)
    return abi.tri_attn_rotary(**args)


@pytest.mark.parametrize("kw,exc", [
    (dict(q=0), ValueError), (dict(positions=0), ValueError), (dict(turns=0), ValueError), (dict(q_out=0), ValueError),
    (dict(k=0), ValueError), (dict(Hk=0), ValueError), (dict(total=-1), ValueError), (dict(Hq=0), ValueError),
    (dict(q=A + 8), ValueError), (dict(k_out=A + 4), ValueError), (dict(turns=A + 4), ValueError),
    (dict(positions=A + 2), ValueError),
    (dict(dtype=abi.TA_E4M3), ValueError), (dict(rotary_dim=63), ValueError), (dict(rotary_dim=66), ValueError),
    (dict(rotary_dim=0), ValueError), (dict(q_row_stride=64), ValueError),
    (dict(q_out=A, q_out_row_stride=512), ValueError),
    (dict(D=264, rotary_dim=8), NotImplementedError), (dict(D=12, rotary_dim=8), NotImplementedError),
    (dict(q_row_stride=260), NotImplementedError),
])
def test_refused(kw, exc):
    with pytest.raises(exc):
        _call(**kw)


def test_no_rows_is_nothing_to_do():
    _call(total=0)


def test_python_refusals():
    import masked_attention_tri_gb300 as ta
    r = ta.Rotary(8)
    q = torch.zeros(3, 2, 8)
    with pytest.raises(ValueError):  # CPU tensors
        ta.rotary_embedding(q, None, torch.zeros(3, dtype=torch.int32), r)
    with pytest.raises(TypeError):
        ta.rotary_embedding([1], None, None, r)


# ---------------------------------------------------------------------------- GPU

CASES = [
    # tokens, Hq, Hk, D, dim, interleaved, dtype, scaling
    (1, 1, 1, 8, 8, False, torch.bfloat16, None),
    (1, 32, 8, 128, 128, False, torch.bfloat16, None),
    (77, 5, 1, 96, 64, True, torch.bfloat16, "yarn"),
    (130, 3, 3, 80, 32, False, torch.float16, "linear"),
    (33, 4, 2, 256, 256, True, torch.float16, "ntk"),
    (64, 2, 2, 72, 6, False, torch.float16, None),      # one pair at a time
    (19, 3, 1, 40, 18, True, torch.bfloat16, None),     # one pair at a time, interleaved
    (50, 2, 1, 20, 12, False, torch.float32, None),     # fp32, one pair at a time
    (401, 6, 2, 64, 64, False, torch.float32, "yarn"),
    (9, 7, 7, 100, 40, True, torch.float32, None),
    (5000, 16, 4, 64, 64, False, torch.bfloat16, None),
]


def _inputs(tokens, Hq, Hk, D, dtype, far=1 << 31):
    g = torch.Generator().manual_seed(tokens * 31 + D)
    q = torch.randn(tokens, Hq, D, generator=g).to(dtype)
    k = torch.randn(tokens, Hk, D, generator=g).to(dtype)
    pos = torch.randint(-1000, 200000, (tokens,), generator=g, dtype=torch.int64)
    pos[0] = far - 1
    if tokens > 2:
        pos[1], pos[2] = -far, 0
    return q, k, pos.to(torch.int32)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,Hq,Hk,D,dim,inter,dtype,scaling", CASES)
@pytest.mark.parametrize("back", [False, True])
def test_values(tokens, Hq, Hk, D, dim, inter, dtype, scaling, back):
    import masked_attention_tri_gb300 as ta
    r = ta.Rotary(dim, interleaved=inter, scaling=scaling, factor=4.0 if scaling else 1.0, original_length=4096,
                  device="cuda")
    q, k, pos = _inputs(tokens, Hq, Hk, D, dtype)
    fn = ta.rotary_embedding_backward if back else ta.rotary_embedding
    gq, gk = fn(q.cuda(), k.cuda(), pos.cuda(), r)
    # theta in fp64 times 2^31 is off by 2^-52 2^31 rad at most: far below the tolerance
    for got, x in ((gq, q), (gk, k)):
        _check(got, *_turn64(x, pos, r, back))
    alone = fn(q.cuda(), None, pos.cuda(), r)
    assert torch.equal(alone, gq)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_views_in_place_and_rows_between(dtype):
    import masked_attention_tri_gb300 as ta
    total, H, D = 70, 4, 64
    r = ta.Rotary(32, device="cuda")
    q, k, pos = _inputs(total, H, H, D, dtype)
    want = ta.rotary_embedding(q.cuda(), k.cuda(), pos.cuda(), r)
    qkv = torch.randn(total, 3, H, D, device="cuda").to(dtype)
    qkv[:, 0], qkv[:, 1] = q.cuda(), k.cuda()
    v = qkv[:, 2].clone()
    a, b, _ = qkv.unbind(1)
    got = ta.rotary_embedding(a, b, pos.cuda(), r, out_q=a, out_k=b)
    assert got[0].data_ptr() == a.data_ptr()
    assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(qkv[:, 2], v)
    with pytest.raises(ValueError):  # rows that overlap
        ta.rotary_embedding(q.cuda()[:1].expand(total, H, D), None, pos.cuda(), r)
    with pytest.raises(ValueError):
        ta.rotary_embedding(q.cuda(), None, pos.cuda().long(), r)
    with pytest.raises(ValueError):  # frequencies on another device
        ta.rotary_embedding(q.cuda(), None, pos.cuda(), ta.Rotary(32))
    empty = ta.rotary_embedding(q.cuda()[:0], k.cuda()[:0], pos.cuda()[:0], r)
    assert empty[0].shape == (0, H, D)


@pytest.mark.gpu
def test_nonfinite_stays_in_its_pair():
    import masked_attention_tri_gb300 as ta
    r = ta.Rotary(16, device="cuda")
    q = torch.zeros(2, 1, 24, device="cuda")
    q[0, 0, 3], q[0, 0, 20] = math.nan, math.inf
    y = ta.rotary_embedding(q, None, torch.tensor([5, 6], dtype=torch.int32, device="cuda"), r)
    bad = {i for i in range(24) if not math.isfinite(float(y[0, 0, i]))}
    assert bad == {3, 11, 20} and float(y[0, 0, 20]) == math.inf and bool(torch.isfinite(y[1]).all())


@pytest.mark.gpu
def test_gradient_against_differences_and_the_formula():
    import masked_attention_tri_gb300 as ta
    r = ta.Rotary(24, interleaved=True, scaling="yarn", factor=2.0, original_length=64, device="cuda")
    q, k, pos = _inputs(6, 2, 1, 32, torch.float32, far=4096)
    q, k, pos = q.cuda().requires_grad_(True), k.cuda().requires_grad_(True), pos.cuda()
    g = torch.Generator().manual_seed(1)
    wq, wk = torch.randn(6, 2, 32, generator=g).cuda(), torch.randn(6, 1, 32, generator=g).cuda()
    loss = lambda a, b: sum((x.double() * w.double()).sum() for x, w in zip(ta.rotary_embedding_autograd(a, b, pos, r), (wq, wk)))  # noqa: E731
    loss(q, k).backward()
    for t, w in ((q, wq), (k, wk)):
        _check(t.grad, *_turn64(w, pos, r, True))
    # differences: the loss is linear in q, so one step of 1 is exact up to the outputs' rounding
    # (two turns of values below 8 in fp32, each off by 8 * 2^-21 at most, weights below 4: 2^-14)
    with torch.no_grad():
        for at in ((0, 0, 0), (1, 1, 17), (5, 0, 31)):
            q2 = q.detach().clone()
            q2[at] += 1
            assert abs(float(loss(q2, k) - loss(q, k)) - float(q.grad[at])) < 2.0 ** -14
    a = torch.randn(6, 2, 32, device="cuda", requires_grad=True)
    ta.rotary_embedding_autograd(a, None, pos, r).sum().backward()  # an expanded gradient
    assert a.grad.shape == a.shape


@pytest.mark.gpu
def test_graph_and_other_stream():
    import masked_attention_tri_gb300 as ta
    r = ta.Rotary(64, device="cuda")
    q, k, pos = (t.cuda() for t in _inputs(40, 4, 2, 64, torch.bfloat16))
    want = ta.rotary_embedding(q, k, pos, r)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = ta.rotary_embedding(q, k, pos, r)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = ta.rotary_embedding(q, k, pos, r)
    q2 = q.flip(0).contiguous()
    q.copy_(q2)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, other))
    assert torch.equal(cap[0], ta.rotary_embedding(q2, None, pos, r)) and torch.equal(cap[1], want[1])
