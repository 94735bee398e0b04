"""Packed attention with a sliding window and first keys that stay visible, forward and backward.

The reference is dense fp64 attention and its gradient formulas, sequence by sequence.
Tolerances.  With u = eps / 2 of the inputs' type (0 for fp32) and per row A = sum_k P |v|: the weights P are rounded
to the type, and the result, so |O - O64| <= u |O| + (u + e) A with e the fp32 arithmetic: logits off by
D 2^-23 E (E the largest sum of |q k| scale behind one) and 2^-22 |x|, twice that on a weight, the sums' n 2^-23, the
exponential's 2^-21.  Backward: P and dx = P (dP - delta) are rounded to the type before the products, delta
comes from the rounded O (u sum |dO O| + the error of O in dO), so with m = P (|dP| + |delta|):
  dV: u |dV| + (u + e) sum_q P |dO|;   dK, dQ: u |dK| + s sum_q (u + 2 e) m |Q| + s sum_q P ddelta |Q|,
  ddelta = sum_d |dO| (u |O| + (u + e) A).
fp16 has a least step of 2^-24, so each rounding to it is off by up to 2^-25 where u |x| is less: f = 2^-25 (0 for
the other types) joins the rounded results and, for each kept pair, the rounded P (relative to the row's largest in the
forward) and dx.
"""
import math

import pytest
import torch

from masked_attention_tri_gb300 import abi, build

A = 0x10000


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


# ---------------------------------------------------------------------------- CPU

def _fwd(**kw):
    args = dict(q=A, k=A, v=A, dtype=abi.TA_BF16, cu_seqlens_q=A, cu_seqlens_k=A, num_seqs=2, total_q=0, total_k=100,
                max_seqlen_q=64, max_seqlen_k=64, H=2, D=64, scale=0.125, kv_num_blocks=0, kv_indices=0,
                full_kv_num_blocks=0, full_kv_indices=0, mask_heads=1, max_q_blocks=1, max_kv_blocks=1, block_q=128,
                block_k=128, mask_mod=abi.TA_MASK_SINK_WINDOW, window=4, prefix_lengths=0, prefix_length=2, bias=0,
                bias_dtype=abi.TA_F32, q_row_stride=0, k_row_stride=0, v_row_stride=0, out=A, lse=0, max_=0, stream=0)
    args.update(kw)
    return abi.tri_attn_varlen_fwd_masked(**args)


def test_refusals():
    import masked_attention_tri_gb300 as ta
    _fwd()
    for kw in (dict(window=0), dict(window=-3), dict(prefix_length=-1), dict(prefix_lengths=A + 2), dict(mask_mod=4),
               dict(mask_mod=5), dict(mask_mod=7)):
        with pytest.raises(ValueError):
            _fwd(**kw)
    bm = ta.BlockMask.from_kv_blocks(torch.zeros(1, 1, 1), torch.zeros(1, 1, 1, 1), mask_mod="sink_window")
    assert bm.mask_mod_code == abi.TA_MASK_SINK_WINDOW
    from masked_attention_tri_gb300.api import _prefix_args
    with pytest.raises(ValueError):
        _prefix_args(None, 1, None, abi.TA_MASK_CAUSAL, 4)
    with pytest.raises(ValueError):
        _prefix_args(3, 1, None, abi.TA_MASK_SINK_WINDOW, 4)
    with pytest.raises(ValueError):
        _prefix_args(None, 1, None, abi.TA_MASK_SINK_WINDOW, -4)


# ---------------------------------------------------------------------------- GPU

def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cu(lens):
    return [sum(lens[:i]) for i in range(len(lens) + 1)]


def _dense(q, k, v, g, lens, lens_k, window, sinks, scale, dtype):
    """fp64 results and tolerances: {name: (value, tolerance)}."""
    u = 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2
    uo = torch.finfo(dtype).eps / 2
    f = 2.0 ** -25 if dtype == torch.float16 else 0.0
    D = q.shape[2]
    res = {n: (torch.zeros(t.shape, dtype=torch.float64), torch.zeros(t.shape, dtype=torch.float64))
           for n, t in (("out", q), ("dq", q), ("dk", k), ("dv", k))}
    lse = (torch.zeros(q.shape[1], q.shape[0], dtype=torch.float64), torch.zeros(q.shape[1], q.shape[0], dtype=torch.float64))
    cq, ck = _cu(lens), _cu(lens_k)
    for i, (n, nk) in enumerate(zip(lens, lens_k)):
        if n == 0 or nk == 0:
            continue
        a, b = slice(cq[i], cq[i + 1]), slice(ck[i], ck[i + 1])
        Q, K, V, G = (x.double().transpose(0, 1) for x in (q[a], k[b], v[b], g[a]))
        s = sinks if isinstance(sinks, int) else sinks[i]
        qi, kj = torch.arange(n)[:, None], torch.arange(nk)
        keep = (kj <= qi) & ((kj > qi - window) | (kj < s))
        x = (Q @ K.transpose(1, 2)) * scale
        E = (Q.abs() @ K.abs().transpose(1, 2)).amax(-1, keepdim=True) * scale
        dx = D * 2.0 ** -23 * E + 2.0 ** -22 * x.abs().amax(-1, keepdim=True)
        e = 2 * dx + nk * 2.0 ** -23 + 2.0 ** -21
        x = x.masked_fill(~keep, -1e9)
        L = torch.logsumexp(x, -1)
        P = torch.softmax(x, -1)
        O = P @ V
        AV = P @ V.abs()
        kept = keep.double().expand_as(P) + (~keep.any(-1, keepdim=True)).double()  # (no valid key: every key counts)
        tO = uo * O.abs() + (u + e) * AV + f + f * P.amax(-1, keepdim=True) * (kept @ V.abs())
        dP = G @ V.transpose(1, 2)
        delta = (G * O).sum(-1, keepdim=True)
        dd = (G.abs() * tO).sum(-1, keepdim=True) + D * 2.0 ** -23 * (G * O).abs().sum(-1, keepdim=True)
        dX = torch.where(keep, P * (dP - delta), torch.zeros(()).double())
        m = torch.where(keep, P * (dP.abs() + delta.abs() + D * 2.0 ** -23 * (G.abs() @ V.abs().transpose(1, 2))), torch.zeros(()).double())
        tX = f * kept + (u + 2 * e) * m + torch.where(keep, P * dd, torch.zeros(()).double())
        T = lambda y: y.transpose(0, 1)  # noqa: E731
        res["out"][0][a], res["out"][1][a] = T(O), T(tO)
        dV = P.transpose(1, 2) @ G
        res["dv"][0][b] = T(dV)
        res["dv"][1][b] = T(f + f * (kept.transpose(1, 2) @ G.abs()) + uo * dV.abs() + ((u + e + n * 2.0 ** -23) * P).transpose(1, 2) @ G.abs())
        dQ, dK = scale * (dX @ K), scale * (dX.transpose(1, 2) @ Q)
        acc = n * 2.0 ** -23 + nk * 2.0 ** -23
        res["dq"][0][a] = T(dQ)
        res["dq"][1][a] = T(f + uo * dQ.abs() + scale * ((tX + acc * m) @ K.abs()))
        res["dk"][0][b] = T(dK)
        res["dk"][1][b] = T(f + uo * dK.abs() + scale * ((tX + acc * m).transpose(1, 2) @ Q.abs()))
        lse[0][:, a] = L
        lse[1][:, a] = torch.where(L < -9e8, torch.full((), 64.0).double(), dx[..., 0] + nk * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -23 * L.abs())
    res["lse"] = lse
    return res


B16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _problem(lens, lens_k, H, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    mk = lambda n: torch.randn(n, H, D, generator=g).to(dtype)  # noqa: E731
    return mk(sum(lens)), mk(sum(lens_k)), mk(sum(lens_k)), mk(sum(lens))


def _run(q, k, v, g, lens, lens_k, window, sinks, scale, **kw):
    import masked_attention_tri_gb300 as ta
    cu, ck = _i32(_cu(lens)), _i32(_cu(lens_k))
    sk = sinks if isinstance(sinks, int) else _i32(sinks)
    mask = dict(window=window, sinks=sk, scale=scale, **(kw if kw else dict(mask_mod="sink_window")))
    q, k, v, g = (x.cuda() for x in (q, k, v, g))
    o, lse, _ = ta.varlen_attention(q, k, v, cu, ck, max(lens), max(lens_k), return_aux=True, **mask)
    dq, dk, dv, _ = ta.varlen_attention_backward(q, k, v, cu, ck, max(lens), max(lens_k), o, lse, g, **mask)
    torch.cuda.synchronize()
    assert ta.get_status() == 0
    return {"out": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _check(got, want, names=("out", "lse", "dq", "dk", "dv")):
    for n in names:
        y, tol = want[n]
        err = (got[n].double().cpu() - y).abs()
        assert bool((err <= tol).all()), (n, float((err - tol).max()), float(err.max()))


CASES = [
    # lens, lens_k (None: the same), H, D, window, sinks
    ([1, 2, 127, 128, 129, 300], None, 2, 64, 64, 4),
    ([700], None, 1, 128, 100, 130),
    ([513, 1, 260], None, 2, 32, 1, 0),
    ([513, 260], None, 1, 96, 1, 1),
    ([400, 77, 640], None, 2, 64, 200, [0, 5, 300]),
    ([300, 140], None, 1, 16, 1000, 3),             # a window wider than the sequences: causal
    ([50, 300, 129], [90, 300, 40], 2, 64, 33, 2),  # fewer and more queries than keys
    ([400, 300], [100, 290], 1, 64, 20, 0),         # queries whose window lies past the keys: none valid
    ([400, 300], [100, 0], 1, 128, 20, 7),          # a sequence without keys
    ([9000], None, 1, 64, 300, 20),                 # more than 64 key blocks
    ([330, 200], None, 2, 80, 90, 10),
    # long sequences beside short ones: the first key blocks are shared by several CTAs
    ([2500, 1, 1400, 128], None, 2, 64, 130, 4),
    ([2100, 700], None, 1, 128, 65, 200),
    ([2100, 1300], None, 1, 64, 100, [3, 0]),
    ([2100, 1300], [1900, 60], 1, 96, 100, 30),
    ([2100], [2100], 1, 32, 1, 400),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [B16, F16, F32])
@pytest.mark.parametrize("lens,lens_k,H,D,window,sinks", CASES)
def test_forward_and_gradients(lens, lens_k, H, D, window, sinks, dtype):
    if dtype == F32 and sum(lens) > 5000:
        lens, window = [1500], 100
    lens_k = lens_k or lens
    q, k, v, g = _problem(lens, lens_k, H, D, dtype, seed=sum(lens) + D)
    s = 1 / math.sqrt(D)
    got = _run(q, k, v, g, lens, lens_k, window, sinks, s)
    want = _dense(q, k, v, g, lens, lens_k, window, sinks, s, dtype)
    if 0 in lens_k:  # no keys: O = 0, lse = -inf; nothing reaches the others
        a = _cu(lens)[lens_k.index(0)]
        assert bool((got["out"][a:a + lens[lens_k.index(0)]] == 0).all()) and bool((got["lse"][:, a:] == -math.inf).all())
        got["lse"] = torch.where(got["lse"] == -math.inf, torch.zeros((), device="cuda"), got["lse"])
    _check(got, want)


def test_workspace_of_shared_key_blocks():
    plain = abi.tri_attn_varlen_bwd_workspace_size(5000, 2, 64, 2500, 2500, False)
    size = lambda *a: abi.tri_attn_varlen_bwd_sink_workspace_size(3, 5000, 2, 64, *a) - plain  # noqa: E731
    assert size(2500, 2500, False, 130, 4) == size(2500, 2500, False, 130, -1) == 3 * 2 * 2 * 128 * 64 * 4
    assert size(2500, 2500, False, 130, 200) == 2 * 3 * 2 * 2 * 128 * 64 * 4
    # many short sequences beside a long one: no accumulator larger than dQ's
    many = lambda S: abi.tri_attn_varlen_bwd_sink_workspace_size(S, 5000, 2, 64, 2500, 2500, False, 130, 4) - plain  # noqa: E731
    assert many(19) == 19 * 2 * 2 * 128 * 64 * 4 and many(20) == 0
    # no sinks, few far blocks, too many first blocks
    assert size(2500, 2500, False, 130, 0) == size(1000, 1000, False, 130, 4) == size(2500, 2500, False, 130, 600) == 0


@pytest.mark.gpu
def test_backward_without_room_for_sharing():
    """The plain workspace is enough: the same gradients up to the order of sums."""
    import masked_attention_tri_gb300 as ta
    from masked_attention_tri_gb300.api import _DT, _stream
    lens, H, D = [2500, 300], 2, 64
    q, k, v, g = (x.cuda() for x in _problem(lens, lens, H, D, B16, seed=21))
    cu = _i32(_cu(lens))
    o, lse, _ = ta.varlen_attention(q, k, v, cu, cu, 2500, 2500, return_aux=True, mask_mod="sink_window", window=130, sinks=4)
    n = abi.tri_attn_varlen_bwd_workspace_size(2800, H, D, 2500, 2500, False)
    ws = torch.full((n // 4 + 4096,), 777.0, device="cuda")
    grads = [torch.empty_like(q) for _ in range(3)]
    abi.tri_attn_varlen_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), _DT[B16], cu.data_ptr(), cu.data_ptr(), 2, 2800, 2800,
                            2500, 2500, H, D, 0.125, 0, 0, 0, 0, 1, 0, 0, 128, 128, abi.TA_MASK_SINK_WINDOW, 130, 0, 4, 0,
                            abi.TA_F32, lse.data_ptr(), o.data_ptr(), g.data_ptr(), *(x.data_ptr() for x in grads), 0,
                            ws.data_ptr(), n, _stream(q.device))
    want = _dense(*(x.cpu() for x in (q, k, v, g)), lens, lens, 130, 4, 0.125, B16)
    _check(dict(zip(("dq", "dk", "dv"), grads)), want, ("dq", "dk", "dv"))
    assert bool((ws[n // 4:] == 777.0).all()) and ta.get_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("D,dtype", [(136, B16), (256, F16)])
def test_wide_heads(D, dtype):
    lens = [200, 333]
    q, k, v, g = _problem(lens, lens, 1, D, dtype, seed=D)
    _check(_run(q, k, v, g, lens, lens, 70, 5, 0.1), _dense(q, k, v, g, lens, lens, 70, 5, 0.1, dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [B16, F32])
def test_equals_the_same_mask_by_other_means(dtype):
    """No sinks: the sliding window; a list of every block: the same rows.  A negative scale, too."""
    import masked_attention_tri_gb300 as ta
    lens = [300, 513]
    q, k, v, g = _problem(lens, lens, 2, 64, dtype, seed=3)
    for scale in (0.125, -0.2):
        want = _dense(q, k, v, g, lens, lens, 64, 0, scale, dtype) if scale > 0 else None
        a = _run(q, k, v, g, lens, lens, 64, 0, scale)
        cu = _i32(_cu(lens))
        b = ta.varlen_attention(q.cuda(), k.cuda(), v.cuda(), cu, cu, 513, 513, scale=scale, mask_mod="sliding_window",
                                window=64, return_aux=True)
        # the kernels add a block of weights that are all 0 in one of the two: equal up to fp32's order of sums
        assert float((a["out"].float() - b[0].float()).abs().max()) <= torch.finfo(dtype).eps * 4
        if want:
            _check(a, want)
    n = torch.tensor([[[3, 3, 3, 0, 0]], [[5, 5, 5, 5, 5]]], dtype=torch.int32, device="cuda")
    idx = torch.arange(5, dtype=torch.int32, device="cuda").expand(2, 1, 5, 5).contiguous()
    bm = ta.BlockMask.from_kv_blocks(n, idx, mask_mod="sink_window")
    got = _run(q, k, v, g, lens, lens, 64, 9, 0.125, block_mask=bm)
    _check(got, _dense(q, k, v, g, lens, lens, 64, 9, 0.125, dtype))


@pytest.mark.gpu
def test_many_sequences():
    """More sequences than the key-split kernel's schedule holds."""
    lens = [3 + (i * 7) % 40 for i in range(1100)]
    q, k, v, g = _problem(lens, lens, 1, 64, B16, seed=1)
    _check(_run(q, k, v, g, lens, lens, 8, 2, 0.125), _dense(q, k, v, g, lens, lens, 8, 2, 0.125, B16))


@pytest.mark.gpu
def test_many_items_of_a_cta():
    """6400 (sequence, head, q block) items, some forty for each CTA: the ring of items goes round several times."""
    import masked_attention_tri_gb300 as ta
    lens, H = [1 + (i * 7) % 40 for i in range(100)], 64
    q, k, v, g = _problem(lens, lens, H, 32, B16, seed=2)
    _check(_run(q, k, v, g, lens, lens, 8, 2, 0.2), _dense(q, k, v, g, lens, lens, 8, 2, 0.2, B16))
    cu = _i32(_cu(lens))
    o, lse, _ = ta.varlen_attention(q.cuda(), k.cuda(), v.cuda(), cu, cu, 40, 40, scale=0.2, mask_mod="causal", return_aux=True)
    torch.cuda.synchronize()
    assert ta.get_status() == 0
    _check({"out": o, "lse": lse}, _dense(q, k, v, g, lens, lens, 1000, 0, 0.2, B16), ("out", "lse"))


@pytest.mark.gpu
def test_bias_and_strided_rows():
    import masked_attention_tri_gb300 as ta
    lens = [300, 129]
    q, k, v, g = _problem(lens, lens, 2, 64, B16, seed=8)
    bias = torch.randn(2, 300, 304, generator=torch.Generator().manual_seed(2)).to(B16)
    cu = _i32(_cu(lens))
    qkv = torch.stack([q, k, v], 1).cuda()
    plain = _run(q, k, v, g, lens, lens, 50, 3, 0.125)
    got = ta.varlen_attention_qkvpacked(qkv, cu, 300, scale=0.125, mask_mod="sink_window", window=50, sinks=3)
    assert torch.equal(got, plain["out"])
    o = ta.varlen_attention(q.cuda(), k.cuda(), v.cuda(), cu, cu, 300, 304, scale=0.125, mask_mod="sink_window",
                            window=50, sinks=3, bias=bias.cuda()).double().cpu()
    t = 0
    for n in lens:
        Q, K, V = (x[t:t + n].double().transpose(0, 1) for x in (q, k, v))
        i, j = torch.arange(n)[:, None], torch.arange(n)
        x = (Q @ K.transpose(1, 2)) * 0.125 + bias[:, :n, :n].double()
        w = x.masked_fill(~((j <= i) & ((j > i - 50) | (j < 3))), -math.inf).softmax(-1)
        # half a step of O and of each weight, and fp32's 64 2^-23 times logits of at most 20
        tol = 2.0 ** -8 * (w @ V).abs() + (2.0 ** -8 + 2.0 ** -12) * (w @ V.abs())
        assert bool(((o[t:t + n].transpose(0, 1) - w @ V).abs() <= tol).all())
        t += n


@pytest.mark.gpu
@pytest.mark.parametrize("D,bias_dtype", [(64, B16), (64, F32), (128, B16), (128, F32), (40, F32)])
def test_gradients_with_a_bias(D, bias_dtype):
    """dBias is the sum over the sequences; tolerances by the forms at the top, the bias being one more exact logit
    term: per row m = P (|dP| + |delta|) and its errors, summed over queries, keys or sequences.  Here with one factor
    for all: every P, dS and result is off by at most u relative to its magnitudes, delta by u sum |dO O|, and
    fp32's own errors (64 logits' units of 2^-23 D) are below u / 8."""
    import masked_attention_tri_gb300 as ta
    lens, H, w, sinks, u = [300, 129, 200], 2, 70, 3, 2.0 ** -8
    q, k, v, g = _problem(lens, lens, H, D, B16, seed=9 + D)
    bias = torch.randn(H, 300, 304, generator=torch.Generator().manual_seed(2)).to(bias_dtype)
    cu, s = _i32(_cu(lens)), 1 / math.sqrt(D)
    dev = [x.cuda() for x in (q, k, v)]
    mask = dict(mask_mod="sink_window", window=w, sinks=sinks, bias=bias.cuda())
    o, lse, _ = ta.varlen_attention(*dev, cu, cu, 300, 304, return_aux=True, **mask)
    got = ta.varlen_attention_backward(*dev, cu, cu, 300, 304, o, lse, g.cuda(), **mask)
    assert ta.get_status() == 0
    dbias, tbias, t = torch.zeros(H, 300, 304).double(), torch.zeros(H, 300, 304).double(), 0
    for n in lens:
        Q, K, V, G = (x[t:t + n].double().transpose(0, 1) for x in (q, k, v, g))
        i, j = torch.arange(n)[:, None], torch.arange(n)
        keep = (j <= i) & ((j > i - w) | (j < sinks))
        P = (s * Q @ K.transpose(1, 2) + bias[:, :n, :n].double()).masked_fill(~keep, -math.inf).softmax(-1)
        O, dP = P @ V, G @ V.transpose(1, 2)
        delta = (G * O).sum(-1, keepdim=True)
        dS = P * (dP - delta)
        tO = 2 * u * (P @ V.abs())
        m = P * ((u + u / 8) * (dP.abs() + delta.abs()) + (G.abs() * tO).sum(-1, keepdim=True))
        want = (s * dS @ K, s * dS.transpose(1, 2) @ Q, P.transpose(1, 2) @ G)
        tols = (s * m @ K.abs(), s * m.transpose(1, 2) @ Q.abs(), (u + u / 8) * P.transpose(1, 2) @ G.abs())
        for name, x, y, tol in zip(("dq", "dk", "dv"), got, want, tols):
            err = (x[t:t + n].double().cpu().transpose(0, 1) - y).abs()
            assert bool((err <= tol + u * y.abs()).all()), (name, n, float((err - tol).max()))
        dbias[:, :n, :n] += dS
        tbias[:, :n, :n] += m
        t += n
    err = (got[3].double().cpu() - dbias).abs()
    assert bool((err <= tbias + u * dbias.abs()).all()), float((err - tbias).max())


@pytest.mark.gpu
@pytest.mark.parametrize("L,D", [(11000, 128), (70000, 64)])
def test_long_sequences(L, D):
    """Hundreds of q blocks, against fp64 over each run of queries and the keys that it sees; tolerances as in
    test_gradients_with_a_bias."""
    w, sinks, u, s = 200, 5, 2.0 ** -8, 1 / math.sqrt(D)
    q, k, v, g = (x.cuda() for x in _problem([L], [L], 1, D, B16, seed=D))
    got = {n: x.double() for n, x in _run(q, k, v, g, [L], [L], w, sinks, s).items()}
    Q, K, V, G = (x[:, 0].double() for x in (q, k, v, g))
    ref = {n: torch.zeros(L, D, dtype=torch.float64, device="cuda") for n in ("out", "dq", "dk", "dv")}
    tol = {n: x.clone() for n, x in ref.items()}
    for a in range(0, L, 1000):
        b = min(L, a + 1000)
        i = torch.arange(a, b, device="cuda")[:, None]
        j = torch.cat((torch.arange(min(sinks, b)), torch.arange(max(sinks, a - w + 1), b))).cuda()
        keep = (j <= i) & ((j > i - w) | (j < sinks))
        P = (s * Q[a:b] @ K[j].t()).masked_fill(~keep, -math.inf).softmax(-1)
        O, dP = P @ V[j], G[a:b] @ V[j].t()
        delta = (G[a:b] * O).sum(-1, keepdim=True)
        dS = P * (dP - delta)
        tO = 2 * u * (P @ V[j].abs())
        m = P * ((u + u / 8) * (dP.abs() + delta.abs()) + (G[a:b].abs() * tO).sum(-1, keepdim=True))
        ref["out"][a:b], tol["out"][a:b] = O, tO + u * O.abs()
        ref["dq"][a:b], tol["dq"][a:b] = s * dS @ K[j], s * m @ K[j].abs()
        for n, x, y in (("dk", s * dS.t() @ Q[a:b], s * m.t() @ Q[a:b].abs()),
                        ("dv", P.t() @ G[a:b], (u + u / 8) * P.t() @ G[a:b].abs())):
            ref[n].index_add_(0, j, x)
            tol[n].index_add_(0, j, y)
    for n in ref:
        err = (got[n][:, 0] - ref[n]).abs()
        assert bool((err <= tol[n] + u * ref[n].abs()).all()), (n, float((err - tol[n]).max()))


@pytest.mark.gpu
def test_counts_beyond_int32():
    lens = [300, 140]
    q, k, v, g = _problem(lens, lens, 2, 64, B16, seed=13)
    want = _dense(q, k, v, g, lens, lens, 1000, 0, 0.125, B16)
    for window, sinks in ((2 ** 31 - 1, 0), (2 ** 32 + 5, 4), (5, 2 ** 33)):
        _check(_run(q, k, v, g, lens, lens, window, sinks, 0.125), want)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_captured_steps_in_two_streams(D):
    """Forward and backward captured once for each of two streams (the first key blocks shared out), replayed at the
    same time with new inputs."""
    import masked_attention_tri_gb300 as ta
    lens, H, w, sinks, s = [2500, 300], 2, 130, 4, 0.1
    mask = dict(mask_mod="sink_window", window=w, sinks=sinks, scale=s)
    cu, steps = _i32(_cu(lens)), []
    for i in range(2):
        x = [t.cuda() for t in _problem(lens, lens, H, D, B16, seed=30 + i)]

        def step():
            o, lse, _ = ta.varlen_attention(*x[:3], cu, cu, 2500, 2500, return_aux=True, **mask)
            return (o, lse) + ta.varlen_attention_backward(*x[:3], cu, cu, 2500, 2500, o, lse, x[3], **mask)[:3]
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = step()
        steps.append((x, stream, graph, out))
    new = [_problem(lens, lens, H, D, B16, seed=40 + i) for i in range(2)]
    for (x, *_), y in zip(steps, new):
        for t, n in zip(x, y):
            t.copy_(n)
    torch.cuda.synchronize()
    for _ in range(3):
        for x, stream, graph, out in steps:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    assert ta.get_status() == 0
    for (x, stream, graph, out), y in zip(steps, new):
        _check(dict(zip(("out", "lse", "dq", "dk", "dv"), out)), _dense(*y, lens, lens, w, sinks, s, B16))


@pytest.mark.gpu
def test_gradient_against_differences():
    """fp32: a central difference of step 2^-6 in fp64 of the formula's loss, and the kernel's gradients."""
    lens = [70, 33]
    q, k, v, g = _problem(lens, lens, 1, 16, F32, seed=5)
    got = _run(q, k, v, g, lens, lens, 9, 2, 0.25)

    def loss(q, k, v):
        return float((_dense(q, k, v, g, lens, lens, 9, 2, 0.25, F32)["out"][0] * g.double()).sum())
    h = 2.0 ** -6
    for name, x in (("dq", 0), ("dk", 1), ("dv", 2)):
        for at in ((0, 0, 3), (69, 0, 0), (71, 0, 15), (40, 0, 7)):
            ab = []
            for sgn in (h, -h):
                t = [q.double(), k.double(), v.double()]
                t[x] = t[x].clone()
                t[x][at] += sgn
                ab.append(loss(*t))
            # a third derivative of at most 64 (inputs of a few units, scale 1/4): h^2 / 6 * 64 < 2^-8
            assert abs((ab[0] - ab[1]) / (2 * h) - float(got[name][at])) < 2.0 ** -8


@pytest.mark.gpu
def test_training_run_with_positions():
    """Rotary positions, sink-window attention and both backwards, against fp64 autograd through the whole chain."""
    import masked_attention_tri_gb300 as ta
    lens, H, D = [150, 40], 2, 64
    q, k, v, g = _problem(lens, lens, H, D, F32, seed=4)
    rot = ta.Rotary(D, scaling="yarn", factor=2.0, original_length=32, device="cuda")
    pos = _i32([i for n in lens for i in range(n)])
    cu = _i32(_cu(lens))
    mask = dict(mask_mod="sink_window", window=30, sinks=4)
    qr, kr = ta.rotary_embedding(q.cuda(), k.cuda(), pos, rot)
    o, lse, _ = ta.varlen_attention(qr, kr, v.cuda(), cu, cu, 150, 150, return_aux=True, **mask)
    dq, dk, dv, _ = ta.varlen_attention_backward(qr, kr, v.cuda(), cu, cu, 150, 150, o, lse, g.cuda(), **mask)
    dq, dk = ta.rotary_embedding_backward(dq, dk, pos, rot)

    qd, kd, vd = (x.double().requires_grad_(True) for x in (q, k, v))
    th = torch.tensor(rot.theta, dtype=torch.float64)
    ang = pos.double().cpu()[:, None] * th
    c, s = (ang.cos() * rot.attention_factor)[:, None], (ang.sin() * rot.attention_factor)[:, None]
    turn = lambda x: torch.cat((x[..., :32] * c - x[..., 32:] * s, x[..., :32] * s + x[..., 32:] * c), -1)  # noqa: E731
    t, total = 0, 0
    for n in lens:
        Q, K, V = (x[t:t + n].transpose(0, 1) for x in (turn(qd), turn(kd), vd))
        i, j = torch.arange(n)[:, None], torch.arange(n)
        w = (Q @ K.transpose(1, 2) / 8).masked_fill(~((j <= i) & ((j > i - 30) | (j < 4))), -math.inf).softmax(-1)
        total = total + ((w @ V).transpose(0, 1) * g[t:t + n].double()).sum()
        t += n
    total.backward()
    for got, ref in ((dq, qd.grad), (dk, kd.grad), (dv, vd.grad)):
        # fp32 throughout: sums of some 1e4 products of at most 2^4 each, 2^-24 apart: 2^-14 of the largest value
        assert float((got.double().cpu() - ref).abs().max()) <= 2.0 ** -14 * float(ref.abs().max())
