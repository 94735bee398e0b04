"""Causal attention of prompts with grouped heads: refusals and the reference on the CPU, values and gradients on the GPU
against fp64.

Tolerances.  For a row's weights w, A = sum w |v| and E = scale max_k sum_d |q_d k_d|: a logit is off by at most dx = D 2^-23 E
(an fp32 sum of D products, truncated at worst) + 2^-21 |x| (its base-2 form, the exponent's argument, a scale folded into it); a weight by 2 dx and the
exponential's 2^-21; on tensor cores weights are rounded to the inputs' type (eps / 2; fp16 has a least step: 2^-25 of the
row's reference weight, which is at most its largest); sums of n weights are off by n 2^-23.  So with
    rel = eps_p / 2 + 2 dx + 2^-21 + n 2^-23,
|O - O64| <= eps / 2 |O| + rel A (+ 2^-25 sum |v| in fp16), |lse - lse64| <= dx + 2^-20 + n 2^-24 + 2^-23 |lse|.
Gradients: P is formed from lse, off by dx + the lse's own error; dP = dO . V by D 2^-23 sum |dO v|; delta = dO . O from the
rounded O by eps / 2 sum |dO O| + D 2^-23 sum |dO O|, and by dO . (O's error) where O is the kernel's.  dS = P (dP - delta) is off by
    e = |dS| (eps_p / 2 + 2 rel_p) + P (err dP + err delta),   rel_p = dx + 2^-20 + n 2^-24 + 2^-23 |lse| + 2^-21,
(+ 2^-25 of a least step in fp16), and dQ, dK, dV by the sums of e |k|, e |q|, (eps_p / 2 + 2 rel_p) P |dO|, plus eps / 2 of
the result and n 2^-23 of the sum of magnitudes.  fp32 and bf16 hold nothing below 2^-126 at full precision, and the
exponential gives 0 there: a weight is off by 2^-126 at most beside all that, dS by 2^-126 (1 + |dP - delta|), a result by 2^-126.
"""
import math

import pytest
import torch

from masked_attention_tri_gb300 import abi, build

A = 0x10000
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _cu(n):
    return [0] + [sum(n[:i + 1]) for i in range(len(n))]


def reference(q, k, v, lq, lk, scale, g=None, out=None):
    """fp64 results and what their tolerances need, sequence by sequence and head by head; `out` is the O whose
    product with dO the gradients use (the kernel's), by default the exact one."""
    Hq, Hk, D = q.shape[1], k.shape[1], q.shape[2]
    grp, dev, W = Hq // Hk, q.device, torch.float64
    cq, ck = _cu(lq), _cu(lk)
    eps = torch.finfo(q.dtype).eps
    eps_p = eps if q.dtype != F32 else 2.0 ** -23
    tiny = 2.0 ** -126
    least = 2.0 ** -25 if q.dtype == F16 else tiny
    R = {"o": torch.zeros(q.shape, dtype=W, device=dev), "lse": torch.full((Hq, q.shape[0]), -math.inf, dtype=W, device=dev)}
    T = {"o": torch.zeros_like(R["o"]), "lse": torch.zeros_like(R["lse"])}
    if g is not None:
        for n, x in (("dq", q), ("dk", k), ("dv", k)):
            R[n], T[n] = torch.zeros(x.shape, dtype=W, device=dev), torch.zeros(x.shape, dtype=W, device=dev)
    for i, (n, m) in enumerate(zip(lq, lk)):
        if not n or not m:
            continue
        qs, ks = slice(cq[i], cq[i + 1]), slice(ck[i], ck[i + 1])
        hide = torch.arange(m, device=dev) > torch.arange(m - n, m, device=dev)[:, None]
        none = hide.all(1)
        for h in range(Hq):
            Q, K, V = q[qs, h].to(W), k[ks, h // grp].to(W), v[ks, h // grp].to(W)
            x = scale * (Q @ K.t())
            E = abs(scale) * (Q.abs() @ K.abs().t()).masked_fill(hide, 0).amax(1)
            x = x.masked_fill(hide, -math.inf)
            lse = torch.logsumexp(x, 1)
            P = torch.where(hide, 0.0, (x - torch.where(none, 0.0, lse)[:, None]).exp())
            big = x.masked_fill(hide, 0).abs().amax(1)
            dx = D * 2.0 ** -23 * E + 2.0 ** -21 * big
            rel = eps_p / 2 + 2 * dx + 2.0 ** -21 + m * 2.0 ** -23
            R["o"][qs, h], R["lse"][h, qs] = P @ V, lse
            seen = (~hide).to(W)
            T["o"][qs, h] = eps / 2 * R["o"][qs, h].abs() + rel[:, None] * (P @ V.abs()) + least * (seen @ V.abs())
            T["lse"][h, qs] = dx + 2.0 ** -20 + m * 2.0 ** -24 + 2.0 ** -23 * torch.where(none, 0.0, lse.abs())
            if g is None:
                continue
            G = g[qs, h].to(W)
            O = R["o"][qs, h]
            dP, delta = G @ V.t(), (G * O).sum(1, keepdim=True)
            dS = P * (dP - delta)
            e_dP = D * 2.0 ** -23 * (G.abs() @ V.abs().t())
            e_delta = D * 2.0 ** -23 * (G.abs() * O.abs()).sum(1, keepdim=True) + (G.abs() * T["o"][qs, h]).sum(1, keepdim=True)
            if out is not None:  # (the O at hand is known: its error is not a bound but a value)
                e_delta = D * 2.0 ** -23 * (G.abs() * O.abs()).sum(1, keepdim=True) + \
                    (G * (out[qs, h].to(W) - O)).sum(1, keepdim=True).abs()
            rel_p = (T["lse"][h, qs] + dx + 2.0 ** -21)[:, None]
            e = dS.abs() * (eps_p / 2 + 2 * rel_p) + P * (e_dP + e_delta) + (least + tiny * (dP - delta).abs()) * seen
            R["dq"][qs, h] = scale * (dS @ K)
            T["dq"][qs, h] = abs(scale) * (e @ K.abs() + (n + m) * 2.0 ** -23 * (dS.abs() @ K.abs()))
            R["dk"][ks, h // grp] += scale * (dS.t() @ Q)
            T["dk"][ks, h // grp] += abs(scale) * (e.t() @ Q.abs() + (n * grp) * 2.0 ** -23 * (dS.abs().t() @ Q.abs()))
            R["dv"][ks, h // grp] += P.t() @ G
            T["dv"][ks, h // grp] += ((eps_p / 2 + 2 * rel_p + n * grp * 2.0 ** -23) * P + least * seen).t() @ G.abs()
    if g is not None:
        for n in ("dq", "dk", "dv"):
            T[n] += eps / 2 * R[n].abs() + least
    return R, T


# ---------------------------------------------------------------------------- CPU

def _fwd(**kw):
    args = dict(q=A, k=A, v=A, dtype=abi.TA_BF16, cu_seqlens_q=A, cu_seqlens_k=A, num_seqs=2, total_q=8, total_k=8,
                max_seqlen_q=4, max_seqlen_k=4, Hq=4, Hk=2, D=64, scale=0.125, q_row_stride=0, k_row_stride=0,
                v_row_stride=0, out=A, lse=A, stream=0)
    args.update(kw)
    return abi.tri_attn_prompt_fwd(**args)


def _bwd(**kw):
    args = dict(q=A, k=A, v=A, dtype=abi.TA_BF16, cu_seqlens_q=A, cu_seqlens_k=A, num_seqs=2, total_q=8, total_k=8,
                max_seqlen_q=4, max_seqlen_k=4, Hq=4, Hk=2, D=64, scale=0.125, q_row_stride=0, k_row_stride=0,
                v_row_stride=0, lse=A, out=A, d_out=A, dq=A, dk=A, dv=A, workspace=A, workspace_bytes=1 << 30, stream=0)
    args.update(kw)
    return abi.tri_attn_prompt_bwd(**args)


BAD = [(dict(q=0), ValueError), (dict(k=0), ValueError), (dict(v=0), ValueError), (dict(out=0), ValueError),
       (dict(cu_seqlens_q=0), ValueError), (dict(cu_seqlens_k=0), ValueError), (dict(num_seqs=0), ValueError),
       (dict(total_q=-1), ValueError), (dict(total_k=-1), ValueError), (dict(max_seqlen_q=-1), ValueError),
       (dict(max_seqlen_k=-1), ValueError), (dict(Hk=3), ValueError), (dict(Hk=0), ValueError), (dict(Hq=0), ValueError),
       (dict(q=A + 8), ValueError), (dict(lse=A + 2), ValueError), (dict(cu_seqlens_k=A + 2), ValueError),
       (dict(dtype=abi.TA_E4M3), ValueError), (dict(dtype=abi.TA_INT4), ValueError), (dict(q_row_stride=128), ValueError),
       (dict(D=72 + 4), NotImplementedError), (dict(D=264), NotImplementedError), (dict(k_row_stride=132), NotImplementedError),
       (dict(total_q=1 << 30), NotImplementedError), (dict(num_seqs=1 << 17), NotImplementedError)]


@pytest.mark.parametrize("kw,exc", BAD)
def test_refused(kw, exc):
    for call in (_fwd, _bwd):
        with pytest.raises(exc):
            call(**kw)


@pytest.mark.parametrize("kw", [dict(lse=0), dict(d_out=0), dict(dq=0), dict(dk=0), dict(dv=0), dict(dv=A + 8),
                                dict(workspace=0), dict(workspace=A + 128), dict(workspace_bytes=100)])
def test_backward_refused(kw):
    with pytest.raises(ValueError):
        _bwd(**kw)


def test_nothing_to_do_and_workspace():
    _fwd(total_q=0)
    _fwd(max_seqlen_q=0)
    _bwd(total_q=0, total_k=0, workspace=0, workspace_bytes=0)
    size = abi.tri_attn_prompt_bwd_workspace_size
    assert size(abi.TA_BF16, 1, 0, 100, 0, 100, 4, 2, 64) == 0 and size(abi.TA_BF16, 1, 100, 100, 100, 100, 4, 3, 64) == 0
    # the rows' dO . O; few key tiles, and the parts of dK and dV are there, too (four row tiles for each CTA of a key tile)
    for dt, D in ((abi.TA_F32, 64), (abi.TA_BF16, 256), (abi.TA_BF16, 64)):
        assert size(dt, 1, 100, 100, 100, 100, 4, 2, D) == 448 * 4
    assert size(abi.TA_BF16, 1, 1000, 1000, 1000, 1000, 4, 2, 64) == (4032 + 4 * 2 * 1000 * 2 * 64) * 4


def test_python_refusals():
    import masked_attention_tri_gb300 as ta
    q, k, cu = torch.zeros(4, 4, 8), torch.zeros(4, 2, 8), torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):  # CPU tensors
        ta.prompt_attention(q, k, k, cu, cu, 4, 4)
    with pytest.raises(TypeError):
        ta.prompt_attention([1], k, k, cu, cu, 4, 4)
    with pytest.raises(ValueError):
        ta.prompt_attention(q[0], k, k, cu, cu, 4, 4)


def test_reference_gradients_are_the_differences():
    """Central differences of the fp64 forward: their error is h^2 / 6 of the third derivative and 2^-53 / h of the sums."""
    torch.manual_seed(3)
    lq, lk = [3, 0, 5], [5, 2, 4]
    q, g = torch.randn(8, 4, 8, dtype=torch.float64), torch.randn(8, 4, 8, dtype=torch.float64)
    k, v = torch.randn(11, 2, 8, dtype=torch.float64), torch.randn(11, 2, 8, dtype=torch.float64)
    R, _ = reference(q, k, v, lq, lk, 0.4, g)
    h = 1e-5
    for name, at in (("dq", 0), ("dk", 1), ("dv", 2)):
        for _ in range(3):
            u = torch.randn((q, k, v)[at].shape, dtype=torch.float64)
            f = [(reference(*[t + s * h * u if i == at else t for i, t in enumerate((q, k, v))], lq, lk, 0.4)[0]["o"] * g).sum()
                 for s in (1, -1)]
            assert abs(float((f[0] - f[1]) / (2 * h) - (R[name] * u).sum())) < 1e-6
    assert bool((R["o"][3] == 0).all()) and bool(torch.isinf(R["lse"][:, 3]).all())  # five queries of four keys


# ---------------------------------------------------------------------------- GPU

def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _inputs(lq, lk, Hq, Hk, D, dtype, seed=0, spread=1.0, extra=0):
    g = torch.Generator(device="cuda").manual_seed(seed + D)
    r = lambda n, h: torch.randn(n, h, D, generator=g, device="cuda")  # noqa: E731
    q, go = (r(sum(lq) + extra, Hq) * spread).to(dtype), r(sum(lq) + extra, Hq).to(dtype)
    k, v = (r(sum(lk) + extra, Hk).to(dtype) for _ in range(2))
    return q, k, v, go


def _within(got, R, T, name):
    err, tol = (got.double() - R[name]).abs(), T[name]
    both = torch.isinf(got.double()) & (got.double() == R[name])
    bad = ~((err <= tol) | both)
    assert not bool(bad.any()), (name, int(bad.sum()), float((err - tol).nan_to_num(9e9).masked_fill(both, 0).max()))


def _run(lq, lk, Hq, Hk, D, dtype, back=True, spread=1.0, seed=0, scale=None):
    import masked_attention_tri_gb300 as ta
    q, k, v, g = _inputs(lq, lk, Hq, Hk, D, dtype, seed, spread)
    a = q, k, v, _i32(_cu(lq)), _i32(_cu(lk)), max(lq), max(lk)
    o, lse = ta.prompt_attention(*a, scale, return_aux=True)
    s = 1 / math.sqrt(D) if scale is None else scale
    s = float(torch.tensor(s, dtype=torch.float32))
    R, T = reference(q, k, v, lq, lk, s)
    _within(o, R, T, "o")
    _within(lse, R, T, "lse")
    if back:
        R, T = reference(q, k, v, lq, lk, s, g, out=o)
        for name, x in zip(("dq", "dk", "dv"), ta.prompt_attention_backward(*a, o, lse, g, scale)):
            _within(x, R, T, name)
    assert ta.get_status() == 0


ODD = [
    # queries and keys of each sequence, Hq, Hk, D, dtype
    ([1], [1], 1, 1, 64, BF),
    ([1], [1], 4, 2, 8, F16),
    ([1, 1, 1], [1, 129, 700], 8, 2, 128, BF),
    ([5, 130, 1], [5, 130, 1], 4, 4, 128, BF),
    ([128, 256], [128, 256], 2, 1, 128, F16),
    ([127, 129, 63], [127, 129, 63], 6, 2, 64, BF),
    ([300], [300], 7, 1, 96, BF),                       # groups of seven: 126 rows of a tile
    ([200, 3], [200, 3], 10, 2, 40, F16),
    ([17, 0, 40], [90, 33, 40], 8, 2, 128, BF),         # no queries; more keys than queries
    ([50, 20, 0], [10, 0, 0], 4, 1, 64, F16),           # rows without a key; no keys; nothing
    ([140], [1000], 3, 1, 128, BF),
    ([64], [64], 128, 1, 64, BF),                       # a token a tile
    ([9], [20], 200, 1, 128, BF),                       # more heads in the group than rows in a tile
    ([33], [70], 132, 2, 64, F16),
    ([40, 70], [40, 100], 4, 2, 256, BF),               # CUDA cores
    ([40, 70], [60, 70], 6, 2, 200, F16),
    ([70, 1, 130], [90, 1, 130], 4, 2, 64, F32),
    ([33], [33], 3, 3, 100, F32),
    ([20], [50], 2, 1, 256, F32),
    ([2000], [2000], 4, 1, 128, BF),
    ([700, 1300], [1500, 1300], 8, 2, 64, F16),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lq,lk,Hq,Hk,D,dtype", ODD)
def test_values_and_gradients(lq, lk, Hq, Hk, D, dtype):
    _run(lq, lk, Hq, Hk, D, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(6))
def test_random_sizes(seed):
    import random
    r = random.Random(seed)
    S = r.choice([1, 3, 9, 40])
    lq = [r.choice([0, 1, r.randint(2, 40), r.randint(41, 400)]) for _ in range(S)]
    lq[0] = max(lq[0], 1)
    lk = [max(0, n + r.choice([0, 0, r.randint(-30, 500)])) for n in lq]
    Hk = r.choice([1, 2, 3])
    _run(lq, lk, Hk * r.choice([1, 2, 3, 4, 5, 8, 16]), Hk, r.choice([16, 64, 72, 128]), r.choice([BF, F16]), seed=seed)


@pytest.mark.gpu
@pytest.mark.parametrize("spread,scale", [(30.0, None), (1.0, 3.0), (1.0, -0.5), (1.0, 0.0), (1e-3, None)])
def test_large_and_other_scales(spread, scale):
    _run([150, 40], [400, 40], 4, 2, 128, BF, spread=spread, scale=scale)
    _run([150, 40], [400, 40], 4, 2, 64, F32, spread=spread, scale=scale)


@pytest.mark.gpu
def test_many_items_of_a_cta():
    _run([130] * 60 + [1] * 200, [260] * 60 + [3] * 200, 16, 8, 64, BF)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF, 128), (F16, 64), (F32, 64)])
def test_strided_rows_and_rows_behind_the_last(dtype, D):
    """Views of one interleaved buffer; rows past the last sequence keep what they hold, and may hold NaN."""
    import masked_attention_tri_gb300 as ta
    Hq, Hk, lq = 4, 2, [37, 150]
    n, g = sum(lq), torch.Generator(device="cuda").manual_seed(5)
    buf = torch.randn(n + 9, Hq + 2 * Hk, D, generator=g, device="cuda").to(dtype)
    buf[n:] = math.nan
    q, k, v = buf[:, :Hq], buf[:, Hq:Hq + Hk], buf[:, Hq + Hk:]
    cu = _i32(_cu(lq))
    out = torch.full((n + 9, Hq, D), 7.0, dtype=dtype, device="cuda")
    o, lse = ta.prompt_attention(q, k, v, cu, cu, max(lq), max(lq), return_aux=True, out=out)
    assert bool((o[n:] == 7).all())
    s = float(torch.tensor(1 / math.sqrt(D), dtype=torch.float32))
    go = torch.randn(n + 9, Hq, D, generator=g, device="cuda").to(dtype)
    go[n:] = math.nan
    R, T = reference(q[:n], k[:n], v[:n], lq, lq, s, go[:n], out=o)
    _within(o[:n], R, T, "o")
    _within(lse[:, :n], R, T, "lse")
    dq, dk, dv = ta.prompt_attention_backward(q, k, v, cu, cu, max(lq), max(lq), o, lse, go)
    for x, name in ((dq, "dq"), (dk, "dk"), (dv, "dv")):
        _within(x[:n], R, T, name)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF, 128), (F32, 64)])
def test_written_rows_only(dtype, D):
    """dq, dk, dv of rows behind the last sequence keep what they hold."""
    import masked_attention_tri_gb300 as ta
    lq, Hq, Hk = [70], 4, 2
    q, k, v, g = _inputs(lq, lq, Hq, Hk, D, dtype, extra=60)
    cu = _i32(_cu(lq))
    o, lse = ta.prompt_attention(q, k, v, cu, cu, 70, 70, return_aux=True)
    dq, dk, dv = (torch.full_like(t, 5.0) for t in (q, k, v))
    code = {BF: abi.TA_BF16, F32: abi.TA_F32}[dtype]
    nb = abi.tri_attn_prompt_bwd_workspace_size(code, 1, q.shape[0], k.shape[0], 70, 70, Hq, Hk, D)
    ws = torch.full((nb,), 255, dtype=torch.uint8, device="cuda")
    p = lambda t: t.data_ptr()  # noqa: E731
    abi.tri_attn_prompt_bwd(p(q), p(k), p(v), code, p(cu), p(cu), 1, q.shape[0], k.shape[0], 70, 70, Hq, Hk, D, D ** -0.5, 0, 0,
                            0, p(lse), p(o), p(g), p(dq), p(dk), p(dv), p(ws), nb, torch.cuda.current_stream().cuda_stream)
    for t in (dq, dk, dv):
        assert bool((t[70:] == 5).all()) and not bool((t[:70] == 5).all())


@pytest.mark.gpu
def test_broken_sequences_are_skipped():
    import masked_attention_tri_gb300 as ta
    q, k, v, g = _inputs([100], [100], 2, 1, 64, BF)
    ta.get_status()
    for cu in ([0, 40, 20], [0, 50, 200], [-5, 40, 100]):
        ta.prompt_attention(q, k, v, _i32(cu), _i32(cu), 100, 100)
        assert ta.get_status() == abi.TA_ERR_DEVICE
    out = torch.full_like(q, 3.0)
    ta.prompt_attention(q, k, v, _i32([0, 60, 100]), _i32([0, 60, 100]), 50, 100, out=out)  # 60 of at most 50
    assert ta.get_status() == abi.TA_ERR_DEVICE
    assert bool((out[:60] == 3).all()) and not bool((out[60:] == 3).any())


@pytest.mark.gpu
def test_the_same_twice_and_autograd():
    import masked_attention_tri_gb300 as ta
    lq, lk = [130, 77], [200, 77]
    q, k, v, g = _inputs(lq, lk, 8, 2, 128, BF)
    a = _i32(_cu(lq)), _i32(_cu(lk)), 130, 200
    o1, o2 = ta.prompt_attention(q, k, v, *a), ta.prompt_attention(q, k, v, *a)
    assert bool((o1 == o2).all())
    qa, ka, va = (t.clone().requires_grad_() for t in (q, k, v))
    o = ta.prompt_attention_autograd(qa, ka, va, *a)
    o.backward(g)
    o, lse = ta.prompt_attention(q, k, v, *a, return_aux=True)
    dq, dk, dv = ta.prompt_attention_backward(q, k, v, *a, o, lse, g)
    assert bool((qa.grad == dq).all()) and bool((ka.grad == dk).all()) and bool((va.grad == dv).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF, 128), (F32, 64)])
def test_captured_and_on_another_stream(dtype, D):
    import masked_attention_tri_gb300 as ta
    lq, lk = [130, 77], [200, 77]
    q, k, v, g = _inputs(lq, lk, 4, 2, D, dtype)
    a = q, k, v, _i32(_cu(lq)), _i32(_cu(lk)), 130, 200
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        o, lse = ta.prompt_attention(*a, return_aux=True)
        d = ta.prompt_attention_backward(*a, o, lse, g)
    for i in range(3):
        q.mul_(0.5)
        o.zero_()
        graph.replay()
        want = ta.prompt_attention(*a)
        R, T = reference(q, k, v, lq, lk, float(torch.tensor(D ** -0.5, dtype=torch.float32)), g, out=o)
        assert bool((o == want).all())
        for x, name in zip(d, ("dq", "dk", "dv")):
            _within(x, R, T, name)
    assert ta.get_status() == 0


@pytest.mark.gpu
def test_two_streams_at_once():
    import masked_attention_tri_gb300 as ta
    lq = [700, 300, 40]
    sets = [_inputs(lq, lq, 8, 2, 128, BF, seed=i) for i in range(2)]
    cu = _i32(_cu(lq))
    want = [ta.prompt_attention(q, k, v, cu, cu, 700, 700) for q, k, v, _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, (q, k, v, _) in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                got[i].append(ta.prompt_attention(q, k, v, cu, cu, 700, 700))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(bool((x == want[i]).all()) for x in got[i])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF, 128), (F32, 64)])
def test_hidden_keys_take_no_part(dtype, D):
    """Infinite keys that a row does not see change nothing in it."""
    import masked_attention_tri_gb300 as ta
    q, k, v, _ = _inputs([200], [200], 2, 1, D, dtype)
    cu = _i32([0, 200])
    want = ta.prompt_attention(q, k, v, cu, cu, 200, 200)
    k2 = k.clone()
    k2[150:] = math.inf
    got = ta.prompt_attention(q, k2, v, cu, cu, 200, 200)
    assert bool((got[:150] == want[:150]).all())


@pytest.mark.gpu
def test_empty():
    import masked_attention_tri_gb300 as ta
    q, k = torch.zeros(0, 4, 64, dtype=BF, device="cuda"), torch.ones(5, 2, 64, dtype=BF, device="cuda")
    o, lse = ta.prompt_attention(q, k, k, _i32([0, 0]), _i32([0, 5]), 0, 5, return_aux=True)
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
    d = ta.prompt_attention_backward(q, k, k, _i32([0, 0]), _i32([0, 5]), 0, 5, o, lse, q)
    assert all(bool((x == 0).all()) for x in d)
    q, k = torch.ones(3, 4, 64, dtype=BF, device="cuda"), torch.zeros(0, 2, 64, dtype=BF, device="cuda")
    o, lse = ta.prompt_attention(q, k, k, _i32([0, 3]), _i32([0, 0]), 3, 0, return_aux=True)
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())
    d = ta.prompt_attention_backward(q, k, k, _i32([0, 3]), _i32([0, 0]), 3, 0, o, lse, q)
    assert bool((d[0] == 0).all()) and d[1].shape == (0, 2, 64)
    assert ta.get_status() == 0
