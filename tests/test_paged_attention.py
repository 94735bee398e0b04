"""Attention over a paged cache: refusals on the CPU, values on the GPU against fp64.

Tolerances, for a row's weights w, A = sum w |v| and E = scale max_k sum_d |q_d k_d| (largest
sum behind a logit): a logit is off by at most dx = D 2^-23 E (an fp32 sum of D products, truncated at worst)
+ 2^-22 |x| (its base-2 form and the exponent's argument); a weight by 2 dx and the exponential's 2^-21; the
weights are rounded to the products' 16-bit type (the cache's; f16 for codes: eps / 2) and summed in
fp32 (len 2^-23).  So |O - O64| <= eps_out / 2 |O| + (eps_p / 2 + 2 dx + 2^-21 + len 2^-23) A, and
|lse - lse64| <= dx + 2^-21 + len 2^-24 + 2^-23 |lse|.  16-bit queries of an 8-bit cache are taken as sums of e4m3 terms
(16 apart, the row's largest magnitude scaled to [2^7, 2^8)): two for bf16, off by half of e4m3's least step
2^-9 in the second, 2^-10 2^-4 = 2^-21 2^7, so 2^-21 of that magnitude at most (three for fp16: less); dx grows by scale 2^-21 max|q| max_k sum |k_d|.
fp16 has a least step of 2^-24: an fp16 output is off by 2^-25 there, and an fp16 weight, which is relative to
the row's largest weight times value scale W, by 2^-25 W: 2^-25 W sum |code| over the slots it sees.
"""
import math

import pytest
import torch

from masked_attention_tri_gb300 import abi, build

A = 0x10000
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


# ---------------------------------------------------------------------------- CPU

def _call(**kw):
    args = dict(q=A, dtype=abi.TA_BF16, cu_seqlens_q=A, kv_lengths=A, page_table=A, num_seqs=2, total_q=8,
                max_seqlen_q=4, Hq=4, Hk=2, D=64, q_row_stride=0, scale=0.125, window=0, sinks=0, k_cache=A, v_cache=A,
                cache_dtype=abi.TA_E4M3, k_scale=A, v_scale=A, num_pages=4, page_size=64, max_pages=2, k_strides=None,
                v_strides=None, out=A, lse=A, workspace=A, workspace_bytes=1 << 30, stream=0)
    args.update(kw)
    return abi.tri_attn_paged_fwd(**args)


@pytest.mark.parametrize("kw,exc", [
    (dict(q=0), ValueError), (dict(out=0), ValueError), (dict(kv_lengths=0), ValueError), (dict(page_table=0), ValueError),
    (dict(workspace=0), ValueError), (dict(workspace=A + 128), ValueError), (dict(workspace_bytes=100), ValueError),
    (dict(cu_seqlens_q=0), ValueError), (dict(num_seqs=0), ValueError), (dict(total_q=-1), ValueError),
    (dict(max_seqlen_q=-1), ValueError), (dict(Hk=3), ValueError), (dict(Hk=0), ValueError), (dict(Hq=0), ValueError),
    (dict(window=-1), ValueError), (dict(sinks=-1), ValueError), (dict(q=A + 8), ValueError), (dict(lse=A + 2), ValueError),
    (dict(k_cache=0), ValueError), (dict(v_cache=A + 4), ValueError), (dict(v_scale=0), ValueError),
    (dict(num_pages=0), ValueError), (dict(max_pages=-1), ValueError), (dict(q_row_stride=128), ValueError),
    (dict(dtype=abi.TA_E4M3), ValueError), (dict(v_strides=abi.strides3([8192, 4096, 0])), ValueError),
    (dict(page_size=24), NotImplementedError), (dict(D=72), NotImplementedError), (dict(D=264), NotImplementedError),
    (dict(cache_dtype=abi.TA_F16, k_scale=0, v_scale=0), NotImplementedError), (dict(q_row_stride=260), NotImplementedError),
    (dict(max_seqlen_q=1 << 30), NotImplementedError), (dict(k_strides=abi.strides3([1 << 41, 4096, 64])), NotImplementedError),
])
def test_refused(kw, exc):
    with pytest.raises(exc):
        _call(**kw)


def test_nothing_to_do_and_workspace():
    _call(total_q=0)
    _call(max_seqlen_q=0)
    assert abi.tri_attn_paged_workspace_size(abi.TA_BF16, 0, 4, 2, 64) == 0
    assert abi.tri_attn_paged_workspace_size(abi.TA_BF16, 1, 4, 3, 64) == 0
    assert abi.tri_attn_paged_workspace_size(abi.TA_BF16, 1, 8, 2, 128) > 0


# ---------------------------------------------------------------------------- GPU

def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Problem:
    """Sequences with `news` newest tokens of `helds` slots, in pages that are scattered over the cache; everything that
    no row sees is NaN, and table entries that no row needs are out of range."""

    def __init__(self, news, helds, Hq, Hk, D, P, dtype, cdtype, window=None, sinks=0, seed=0, spread=1.0, extra_rows=0,
                 poison=True):
        g = torch.Generator().manual_seed(seed)
        S, MP = len(news), max(1, max(-(-h // P) for h in helds) + 1)
        self.news, self.helds, self.window, self.sinks, self.P = news, helds, window, sinks, P
        self.Hq, self.Hk, self.D, self.dtype, self.cdtype = Hq, Hk, D, dtype, cdtype
        total = sum(news)
        self.q = (torch.randn(total + extra_rows, Hq, D, generator=g) * spread).to(dtype)
        pages = sum(-(-h // P) for h in helds) + 2
        order = torch.randperm(pages, generator=g).tolist()
        table = [[(-5 if (i + j) % 2 else pages + 7) for j in range(MP)] for i in range(S)]
        self.k = torch.full((pages, Hk, P, D), math.nan, dtype=torch.float64)
        self.v = torch.full((pages, Hk, P, D), math.nan, dtype=torch.float64)
        codes = cdtype == F8
        self.ks = torch.full((pages, Hk), math.nan)
        self.vs = torch.full((pages, Hk), math.nan)
        self.seen = []
        for i, (n, h) in enumerate(zip(news, helds)):
            pos = torch.arange(h - n, h)[:, None]
            j = torch.arange(h)
            see = j <= pos
            if window:
                see = see & ((pos - j < window) | (j < sinks))
            self.seen.append(see)
            any_ = see.any(0)
            for lp in range(-(-h // P)):
                vis = any_[lp * P:(lp + 1) * P]
                if not bool(vis.any()) and poison:
                    continue
                page = table[i][lp] = order.pop()
                sl = torch.nonzero(vis).flatten() if poison else torch.arange(len(vis))
                for x, sc in ((self.k, self.ks), (self.v, self.vs)):
                    rows = torch.randn(Hk, len(sl), D, generator=g)
                    if codes:
                        s = torch.exp2(torch.randint(-8, -4, (Hk,), generator=g).float())
                        sc[page] = s
                        x[page][:, sl] = (rows * 100).clamp(-448, 448).to(F8).double()  # (beyond 448 torch gives NaN)
                    else:
                        x[page][:, sl] = rows.to(cdtype).double()
        self.table = table

    def cache(self, layout=""):
        import masked_attention_tri_gb300 as ta
        k, v = self.k.float().to(self.cdtype).cuda(), self.v.float().to(self.cdtype).cuda()
        if layout == "heads last":
            k, v = (x.view(torch.uint8).view(*x.shape[:3], -1).transpose(1, 2).contiguous().transpose(1, 2).view(self.cdtype)
                    for x in (k, v))
        elif layout == "one buffer":
            k, v = torch.stack([k.view(torch.uint8), v.view(torch.uint8)], 1).view(self.cdtype).unbind(1)
        sc = (self.ks.cuda(), self.vs.cuda()) if self.cdtype == F8 else (None, None)
        return ta.PagedKVCache(k, v, *sc)

    def run(self, layout="", q=None, out=None):
        import masked_attention_tri_gb300 as ta
        one = all(n == 1 for n in self.news) and self.q.shape[0] == len(self.news)
        cu = [0]
        for n in self.news:
            cu.append(cu[-1] + n)
        args = () if one else (_i32(cu), max(max(self.news), 1))
        r = ta.paged_attention(self.q.cuda() if q is None else q, self.cache(layout), _i32(self.table), _i32(self.helds),
                               *args, window=self.window, sinks=self.sinks, return_aux=True, out=out)
        torch.cuda.synchronize()
        assert ta.get_status() == 0
        return r

    def check(self, out, lse):
        G, t0 = self.Hq // self.Hk, 0
        scale = 1 / math.sqrt(self.D)
        eps_p = 0.0 if self.dtype == torch.float32 else torch.finfo(torch.float16 if self.cdtype == F8 else self.cdtype).eps
        eps_o = torch.finfo(self.dtype).eps
        out, lse = out.double().cpu(), lse.double().cpu()
        for i, (n, h) in enumerate(zip(self.news, self.helds)):
            see = self.seen[i]
            cols = torch.nonzero(see.any(0)).flatten() if n else torch.zeros(0, dtype=torch.int64)
            if n and not len(cols):
                assert bool((out[t0:t0 + n] == 0).all()) and bool((lse[:, t0:t0 + n] == -math.inf).all())
            if n and len(cols):
                page = torch.tensor(self.table[i])[cols // self.P]
                kv = []
                for x, sc in ((self.k, self.ks), (self.v, self.vs)):
                    y = x[page, :, cols % self.P]
                    kv.append(y * sc[page].double()[..., None] if self.cdtype == F8 else y)
                k, v = (y.transpose(0, 1).repeat_interleave(G, 0) for y in kv)   # (Hq, keys, D)
                q = self.q[t0:t0 + n].double().transpose(0, 1)                   # (Hq, n, D)
                x = q @ k.transpose(1, 2) * scale
                E = (q.abs() @ k.abs().transpose(1, 2) * scale).amax(-1)
                big = x.abs().amax(-1)
                x = x.masked_fill(~see[:, cols], -math.inf)
                L = torch.logsumexp(x, -1)
                empty = ~see[:, cols].any(-1)
                w = torch.where(empty[None, :, None], torch.zeros(()).double(), (x - L[..., None]).exp())
                o, aa = w @ v, w @ v.abs()
                dx = self.D * 2.0 ** -23 * E + 2.0 ** -22 * big
                if self.cdtype == F8:
                    dx = dx + 2.0 ** -21 * scale * q.abs().amax(-1) * k.abs().sum(-1).amax(-1, keepdim=True)
                tol = eps_o / 2 * o.abs() + (eps_p / 2 + 2 * dx + 2.0 ** -21 + h * 2.0 ** -23)[..., None] * aa
                if self.dtype == torch.float16:
                    tol = tol + 2.0 ** -25
                if self.dtype != torch.float32 and (self.cdtype == F8 or self.cdtype == torch.float16):
                    vs = self.vs[page].double().t().repeat_interleave(G, 0)[:, None] if self.cdtype == F8 else torch.ones(1, 1, 1).double()
                    code = v / vs.transpose(1, 2)
                    tol = tol + 2.0 ** -25 * (w * vs).amax(-1, keepdim=True) * code.abs().sum(1, keepdim=True)
                err = (out[t0:t0 + n].transpose(0, 1) - o).abs()
                assert bool((err <= tol).all()), (i, float((err - tol).max()), float(err.max()))
                gl = lse[:, t0:t0 + n]
                assert bool((gl[:, empty] == -math.inf).all())
                lt = (dx + 2.0 ** -21 + h * 2.0 ** -24 + 2.0 ** -23 * L.abs())[:, ~empty]
                el = (gl - L).abs()[:, ~empty]
                assert bool((el <= lt).all()), (i, float((el - lt).max()))
            t0 += n


B16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
PAIRS = [(B16, F8), (F16, F8), (F32, F8), (B16, B16), (F16, F16), (F32, F32)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,cdtype", PAIRS)
@pytest.mark.parametrize("Hq,Hk,D,P", [(8, 1, 128, 64), (4, 4, 64, 16), (6, 2, 80, 32), (32, 2, 96, 128), (3, 1, 16, 16),
                                       (16, 2, 256, 64), (5, 1, 192, 1024), (40, 1, 128, 16), (36, 1, 256, 32)])
def test_single_tokens(dtype, cdtype, Hq, Hk, D, P):
    """One token of each sequence; lengths around tiles and pages, nothing held, and one long."""
    helds = [1, 0, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 1000, 2500]
    pr = Problem([1] * len(helds), helds, Hq, Hk, D, P, dtype, cdtype, seed=D + P)
    pr.check(*pr.run())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,cdtype", PAIRS)
@pytest.mark.parametrize("Hq,Hk,D,P,window,sinks", [(8, 2, 64, 16, 1, 0), (4, 1, 128, 64, 100, 4), (8, 1, 128, 32, 64, 64),
                                                    (2, 2, 96, 16, 33, 1), (16, 1, 64, 128, 7, 200), (4, 4, 256, 16, 500, 3)])
def test_windows_and_first_slots(dtype, cdtype, Hq, Hk, D, P, window, sinks):
    helds = [1, 5, 64, 65, 100, 101, 300, 1029, 2049]
    pr = Problem([1] * len(helds), helds, Hq, Hk, D, P, dtype, cdtype, window=window, sinks=sinks, seed=window)
    pr.check(*pr.run())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,cdtype", PAIRS)
@pytest.mark.parametrize("Hq,Hk,D,P,window,sinks", [(8, 2, 64, 16, None, 0), (4, 1, 128, 64, 60, 5), (3, 3, 80, 32, 16, 0),
                                                    (24, 2, 96, 64, None, 0)])
def test_several_tokens(dtype, cdtype, Hq, Hk, D, P, window, sinks):
    """Ragged numbers of new tokens (none, one, some, a whole prompt), rows behind the last sequence."""
    news, helds = [5, 0, 1, 70, 130, 2, 0, 9], [5, 40, 129, 70, 200, 2, 0, 1033]
    pr = Problem(news, helds, Hq, Hk, D, P, dtype, cdtype, window=window, sinks=sinks, seed=7, extra_rows=3, poison=False)
    out = torch.full((sum(news) + 3, Hq, D), 9.0, dtype=dtype, device="cuda")
    o, lse = pr.run(out=out)
    assert o is out and bool((out[sum(news):] == 9.0).all())
    pr.check(o, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,cdtype", [(B16, F8), (F16, F16), (F32, F32)])
def test_many_sequences_and_one_long_one(dtype, cdtype):
    g = torch.Generator().manual_seed(3)
    helds = torch.randint(0, 90, (700,), generator=g).tolist()
    helds[431] = 9000
    pr = Problem([1] * 700, helds, 4, 2, 64, 16, dtype, cdtype, seed=11)
    pr.check(*pr.run())


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["heads last", "one buffer"])
@pytest.mark.parametrize("dtype,cdtype", PAIRS)
def test_views(layout, dtype, cdtype):
    """Strided caches and queries give the contiguous result, bit for bit."""
    pr = Problem([1, 1, 1], [70, 129, 300], 8, 2, 64, 32, dtype, cdtype, seed=5, poison=False)
    want = pr.run()
    qkv = torch.randn(3, 3 * 8 * 64, device="cuda").to(dtype)
    q = qkv[:, 512:1024].view(3, 8, 64)
    q.copy_(pr.q)
    got = pr.run(layout, q=q)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    pr.check(*got)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,cdtype", PAIRS)
def test_large_logits_and_uneven_scales(dtype, cdtype):
    """Peaked rows; pages whose scales are far apart (the value scales' exponents too)."""
    pr = Problem([1, 1, 3], [500, 40, 260], 4, 1, 64, 16, dtype, cdtype, seed=9, spread=20.0, poison=False)
    if cdtype == F8:
        g = torch.Generator().manual_seed(1)
        pr.vs = torch.exp2(torch.randint(-40, 20, pr.vs.shape, generator=g).float())
        pr.vs[::3] *= 1.3
        pr.ks = pr.ks * 1.1
        # codes of zero with a huge scale next to values of ordinary size
        pr.v[pr.table[0][2]] = 0
        pr.vs[pr.table[0][2]] = 2.0 ** 50
    pr.check(*pr.run())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,cdtype", PAIRS)
def test_nan_is_seen_where_it_counts(dtype, cdtype):
    """A NaN key of one sequence makes that sequence's rows NaN and no others."""
    pr = Problem([1, 1], [65, 65], 2, 1, 64, 16, dtype, cdtype, seed=2, poison=False)
    pr.k[pr.table[1][0], 0, 3, 5] = math.nan
    o, lse = pr.run()
    assert bool(o[1].isnan().all()) and bool(lse[:, 1].isnan().all())
    assert bool(o[0].isfinite().all()) and bool(lse[:, 0].isfinite().all())
    pr = Problem([1], [1], 2, 1, 64, 16, dtype, cdtype, seed=2, poison=False)
    pr.k[pr.table[0][0], 0, 0, 5] = math.nan
    o, lse = pr.run()
    assert bool(o.isnan().all()) and bool(lse.isnan().all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,cdtype", PAIRS)
def test_broken_contracts(dtype, cdtype):
    import masked_attention_tri_gb300 as ta
    pr = Problem([1, 1], [40, 40], 2, 1, 64, 16, dtype, cdtype, seed=2, poison=False)
    cache, q = pr.cache(), pr.q.cuda()
    good, _ = pr.run()
    call = lambda table, helds, *a: ta.paged_attention(q, cache, _i32(table), _i32(helds), *a, return_aux=True)  # noqa: E731
    # a page out of range: its slots are not seen; the other sequence is as it was
    bad = [row[:] for row in pr.table]
    bad[0][1] = cache.num_pages
    o, _ = call(bad, [40, 40])
    assert ta.get_status() == abi.TA_ERR_DEVICE
    assert torch.equal(o[1], good[1]) and bool(o[0].isfinite().all()) and not torch.equal(o[0], good[0])
    for held in (-1, 16 * len(pr.table[0]) + 1, 2 ** 31 - 1, -2 ** 31):
        o, lse = call(pr.table, [held, 40])
        assert ta.get_status() == abi.TA_ERR_DEVICE and bool((o[0] == 0).all()) and bool((lse[:, 0] == -math.inf).all())
        assert torch.equal(o[1], good[1])
    for cu, most in (([0, 2, 1], 2), ([0, 1, 3], 2), ([-1, 1, 2], 2), ([0, 2, 2], 1)):
        call(pr.table, [40, 40], _i32(cu), most)
        assert ta.get_status() == abi.TA_ERR_DEVICE
    assert ta.get_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,cdtype", [(B16, F8), (F16, F16), (F32, F32)])
def test_replays_streams_and_repeats(dtype, cdtype):
    """The same result every time, on another stream, and from two captured graphs in flight with their own scratch."""
    import masked_attention_tri_gb300 as ta
    pr = Problem([1] * 3, [700, 3000, 90], 8, 2, 64, 16, dtype, cdtype, seed=6, poison=False)
    want = pr.run()
    cache, table, q = pr.cache(), _i32(pr.table), pr.q.cuda()
    held = _i32(pr.helds)
    streams, graphs, outs = [torch.cuda.Stream() for _ in range(2)], [], []
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            a = ta.paged_attention(q, cache, table, held, return_aux=True)
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(a, want))
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                outs.append(ta.paged_attention(q, cache, table, held, return_aux=True))
            graphs.append(graph)
    for _ in range(20):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for o in outs for x, y in zip(o, want))
    held.copy_(_i32([65, 0, 90]))  # other lengths in the same graph
    pr2 = Problem([1] * 3, [700, 3000, 90], 8, 2, 64, 16, dtype, cdtype, seed=6, poison=False)
    pr2.helds, pr2.seen = [65, 0, 90], [torch.ones(1, n, dtype=torch.bool) for n in (65, 0, 90)]
    torch.cuda.synchronize()
    graphs[0].replay()
    torch.cuda.synchronize()
    pr2.check(*outs[0])
    assert ta.get_status() == 0


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    """Pages whose elements lie beyond 2^31 (and bytes beyond 2^32) in a 16-bit cache."""
    import masked_attention_tri_gb300 as ta
    pages, Hk, P, D = 8200, 8, 128, 256
    cache = ta.PagedKVCache(torch.zeros(pages, Hk, P, D, dtype=B16, device="cuda"),
                            torch.zeros(pages, Hk, P, D, dtype=B16, device="cuda"))
    pr = Problem([1], [200], 8, Hk, D, P, B16, B16, seed=8, poison=False)
    at = [pages - 1, pages - 2]
    for lp, page in enumerate(at):
        cache.k[page] = pr.k[pr.table[0][lp]].nan_to_num().to(B16).cuda()
        cache.v[page] = pr.v[pr.table[0][lp]].nan_to_num().to(B16).cuda()
    o, lse = ta.paged_attention(pr.q.cuda(), cache, _i32([at]), _i32([200]), return_aux=True)
    pr.check(o, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("cdtype", [F8, B16])
def test_windows_beyond_int32(cdtype):
    """A window past int32 is every slot, as are sinks past it."""
    import masked_attention_tri_gb300 as ta
    pr = Problem([1, 1], [300, 77], 4, 2, 64, 16, B16, cdtype, seed=4, poison=False)
    want, cache = pr.run(), pr.cache()
    for window, sinks in ((2 ** 31 - 1, 0), (2 ** 32 + 5, 0), (5, 2 ** 32 + 3), (2 ** 40, 2 ** 40)):
        got = ta.paged_attention(pr.q.cuda(), cache, _i32(pr.table), _i32(pr.helds), window=window, sinks=sinks,
                                 return_aux=True)
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("cdtype", [F8, B16])
def test_serving_run(cdtype):
    """A prompt, a chunk and single tokens through append and attention, as a server runs them, against
    fp64 attention over the rows that the cache holds."""
    import masked_attention_tri_gb300 as ta
    from test_rotary import _turn64
    S, Hq, Hk, D, P, MP = 3, 8, 2, 64, 32, 8
    g = torch.Generator().manual_seed(12)
    cache = ta.PagedKVCache.empty(S * MP, Hk, P, D, cdtype)
    table = torch.randperm(S * MP, generator=g).view(S, MP)
    rot = ta.Rotary(D, scaling="yarn", factor=4.0, original_length=64, device="cuda")
    held = [0] * S
    for new in ([50, 1, 90], [7, 64, 0], [1, 1, 1], [1, 1, 1]):
        held = [h + n for h, n in zip(held, new)]
        total = sum(new)
        q, k, v = (torch.randn(total, h, D, generator=g).to(B16) for h in (Hq, Hk, Hk))
        cu = _i32([sum(new[:i]) for i in range(S + 1)])
        args = () if new == [1] * S else (cu, max(new))
        qr = ta.kv_cache_append(cache, k.cuda(), v.cuda(), _i32(table.tolist()), _i32(held), *args, rotary=rot, q=q.cuda())
        o, lse = ta.paged_attention(qr, cache, _i32(table.tolist()), _i32(held), *args, window=40, sinks=2, return_aux=True)
        torch.cuda.synchronize()
        assert ta.get_status() == 0
        pos = torch.cat([torch.arange(h - n, h) for n, h in zip(new, held)])
        want_q, mag = _turn64(q, pos, rot)
        assert bool(((qr.double().cpu() - want_q).abs() <= 2.0 ** -8 * want_q.abs() + mag * 2.0 ** -21).all())
        pr = Problem(new, held, Hq, Hk, D, P, B16, cdtype, window=40, sinks=2, poison=False)
        pr.table, pr.q = table.tolist(), qr.cpu()
        pr.k, pr.v = cache.k.float().double().cpu(), cache.v.float().double().cpu()
        if cdtype == F8:
            pr.ks, pr.vs = cache.k_scale.cpu(), cache.v_scale.cpu()
        pr.check(o, lse)
