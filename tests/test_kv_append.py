"""Appending to a paged cache: refusals on the CPU; rows, codes, scales and what stays untouched on the GPU.

The reference walks sequences, pages and heads in fp64.  16-bit and fp32 caches hold the
turned rows exactly as rotary_embedding gives them.  8-bit codes: v, which is not
turned, has to match the nearest code bit for bit after one append; a value x that may have been
re-coded is off by at most half a step of its first rounding (2^-4 |x|, or 2^-10 scale
below the least normal code) and 2^-10 scale for each later scale (each at least twice the one
before: 2 * 2^-10 of the last in all), plus the turn's fp32 arithmetic (|a| + |b|) m 2^-21.
"""
import math

import pytest
import torch

from masked_attention_tri_gb300 import abi, build
from test_rotary import _turn64

A = 0x10000


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


# ---------------------------------------------------------------------------- CPU

def _call(**kw):
    args = dict(q=A, k=A, v=A, dtype=abi.TA_BF16, cu_seqlens=A, kv_lengths=A, page_table=A, num_seqs=2, total=8,
                max_seqlen=4, Hq=4, Hk=2, D=64, q_row_stride=0, k_row_stride=0, v_row_stride=0, q_out_row_stride=0,
                positions=0, turns=A, rotary_dim=64, interleaved=0, mscale=1.0, k_cache=A, v_cache=A,
                cache_dtype=abi.TA_E4M3, k_scale=A, v_scale=A, num_pages=4, page_size=64, max_pages=2, k_strides=None,
                v_strides=None, q_out=A, stream=0)
    args.update(kw)
    return abi.tri_attn_kv_append(**args)


@pytest.mark.parametrize("kw,exc", [
    (dict(k=0), ValueError), (dict(v=0), ValueError), (dict(kv_lengths=0), ValueError), (dict(page_table=0), ValueError),
    (dict(q=0), ValueError), (dict(q_out=0), ValueError), (dict(Hq=0), ValueError),
    (dict(turns=0), ValueError), (dict(turns=0, rotary_dim=0), ValueError),  # q without a rotation
    (dict(turns=0, rotary_dim=0, q=0, q_out=0, Hq=0, positions=A), ValueError),
    (dict(k_cache=0), ValueError), (dict(k_scale=0), ValueError), (dict(cache_dtype=abi.TA_BF16), ValueError),
    (dict(cu_seqlens=0), ValueError), (dict(num_seqs=0), ValueError), (dict(total=-1), ValueError),
    (dict(max_seqlen=-1), ValueError), (dict(num_pages=0), ValueError), (dict(max_pages=0), ValueError),
    (dict(k_cache=A + 8), ValueError), (dict(k_scale=A + 2), ValueError), (dict(k=A + 2), ValueError),
    (dict(rotary_dim=65), ValueError), (dict(rotary_dim=66), ValueError), (dict(k_row_stride=64), ValueError),
    (dict(dtype=abi.TA_E4M3), ValueError), (dict(cache_dtype=9), ValueError),
    (dict(k_strides=abi.strides3([8192, 4096, 32])), ValueError),
    (dict(k_strides=abi.strides3([8192, 4096, 72])), NotImplementedError),
    (dict(cache_dtype=abi.TA_F16, k_scale=0, v_scale=0), NotImplementedError),
    (dict(page_size=8), NotImplementedError), (dict(page_size=48), NotImplementedError),
    (dict(page_size=2048), NotImplementedError), (dict(D=72, rotary_dim=64), NotImplementedError),
    (dict(D=264), NotImplementedError), (dict(v_row_stride=132), NotImplementedError),
])
def test_refused(kw, exc):
    with pytest.raises(exc):
        _call(**kw)


def test_nothing_to_do():
    _call(total=0)
    _call(max_seqlen=0)


def test_cache_handle_refusals():
    import masked_attention_tri_gb300 as ta
    k = torch.zeros(3, 2, 16, 32)
    ta.PagedKVCache(k, k.clone())
    for bad in (lambda: ta.PagedKVCache(k[0], k[0]), lambda: ta.PagedKVCache(k, k[:2]),
                lambda: ta.PagedKVCache(k, k, torch.zeros(3, 2), torch.zeros(3, 2)),
                lambda: ta.PagedKVCache(k.transpose(2, 3), k.transpose(2, 3))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        ta.PagedKVCache(k.double(), k.double())
    c = k.to(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        ta.PagedKVCache(c, c, torch.zeros(3, 1), torch.zeros(3, 2))
    with pytest.raises(ValueError):  # CPU rows
        ta.kv_cache_append(ta.PagedKVCache(k, k.clone()), torch.zeros(1, 2, 32), torch.zeros(1, 2, 32),
                           torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


# ---------------------------------------------------------------------------- GPU

def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _scale64(most):
    return 2.0 ** min(56, max(-56, math.ceil(math.log2(most / 448)))) if most > 0 else 2.0 ** -56


class Model:
    """The cache as the definition has it: fp64 rows and scales of each (page, head)."""

    def __init__(self, pages, heads, P):
        self.rows, self.scale, self.P = {}, {}, P

    def append(self, table, held, rows, codes):
        """rows (n, Hk, D) fp64 of one sequence whose slots end at `held`."""
        n = rows.shape[0]
        for i in range(n):
            slot = held - n + i
            self.rows[(int(table[slot // self.P]), slot % self.P)] = rows[i]
        if codes:
            for lp in sorted({(held - n + i) // self.P for i in range(n)}):
                lo, hi = max(held - n, lp * self.P), min(held, (lp + 1) * self.P)
                new = rows[lo - held + n:hi - held + n].abs().amax((0, 2))
                for h in range(rows.shape[1]):
                    key = (int(table[lp]), h)
                    s = _scale64(float(new[h]))
                    self.scale[key] = max(s, self.scale[key]) if lo % self.P else s


def _filled(pages, Hk, P, D, dtype, strided):
    """A cache full of a pattern, so that what is left alone can be told."""
    import masked_attention_tri_gb300 as ta
    bytes_ = torch.tensor([], dtype=dtype).element_size()
    if strided == "heads last":
        buf = torch.full((2, pages, P, Hk, D * bytes_), 0x35, dtype=torch.uint8, device="cuda").view(dtype)
        k, v = (b.transpose(1, 2) for b in buf)
    elif strided == "one buffer":
        buf = torch.full((pages, 2, Hk, P, D * bytes_), 0x35, dtype=torch.uint8, device="cuda").view(dtype)
        k, v = buf.unbind(1)
    else:
        k, v = (torch.full((pages, Hk, P, D * bytes_), 0x35, dtype=torch.uint8, device="cuda").view(dtype)
                for _ in range(2))
    sc = [torch.full((pages, Hk), 0.5, device="cuda") for _ in range(2)] if dtype == torch.float8_e4m3fn else [None] * 2
    return ta.PagedKVCache(k, v, *sc)


CASES = [
    # dtype, cache dtype, Hq, Hk, D, dim, interleaved, P, layout
    (torch.bfloat16, torch.float8_e4m3fn, 4, 2, 64, 64, False, 16, ""),
    (torch.bfloat16, torch.float8_e4m3fn, 9, 9, 128, 128, False, 64, "one buffer"),
    (torch.float16, torch.float8_e4m3fn, 2, 1, 96, 32, True, 32, "heads last"),
    (torch.float32, torch.float8_e4m3fn, 3, 1, 48, 36, False, 16, ""),     # one pair at a time
    (torch.float16, torch.float8_e4m3fn, 1, 1, 256, 256, True, 128, ""),
    (torch.float16, torch.float8_e4m3fn, 3, 2, 192, 192, True, 64, ""),    # 64 rows' table: just 48 KB
    (torch.bfloat16, torch.bfloat16, 2, 1, 192, 192, False, 64, ""),
    (torch.bfloat16, torch.float8_e4m3fn, 2, 1, 200 + 8, 96, False, 1024, ""),
    (torch.bfloat16, torch.bfloat16, 8, 2, 72, 40, False, 16, "heads last"),
    (torch.float16, torch.float16, 5, 5, 64, 64, True, 32, "one buffer"),
    (torch.float32, torch.float32, 2, 2, 20, 20, False, 16, ""),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,cdtype,Hq,Hk,D,dim,inter,P,layout", CASES)
def test_rounds_of_appends(dtype, cdtype, Hq, Hk, D, dim, inter, P, layout):
    """A prompt, a short continuation and single tokens, with scales that grow, shrink and start anew."""
    import masked_attention_tri_gb300 as ta
    codes = cdtype == torch.float8_e4m3fn
    g = torch.Generator().manual_seed(D + P)
    S, MP = 4, 6
    pages = S * MP + 2
    table = torch.randperm(pages, generator=g)[:S * MP].view(S, MP)
    cache, model = _filled(pages, Hk, P, D, cdtype, layout), {x: Model(pages, Hk, P) for x in "kv"}
    untouched = {x: getattr(cache, x).view(torch.uint8 if codes else cdtype).clone() for x in "kv"}
    rot = ta.Rotary(dim, interleaved=inter, scaling="yarn", factor=2.0, original_length=64, device="cuda")
    held = [0] * S
    news = [[2 * P + 3, 1, 0, P], [1, P - 1, 5, 0], [1] * S, [1] * S, [3, 0, 2 * P, 1]]
    for step, new in enumerate(news):
        held = [h + n for h, n in zip(held, new)]
        total = sum(new) + 2  # two rows behind the last sequence
        q, k, v = (torch.randn(total, h, D, generator=g) * f for h, f in ((Hq, 1.0), (Hk, 1.0), (Hk, 1.0)))
        grow = [1.0, 40.0, 0.01, 3000.0, 7.0][step]
        k, v = k * grow, v * grow
        v[:, :, 3] = 0
        q, k, v = q.to(dtype), k.to(dtype), v.to(dtype)
        cu = torch.cumsum(torch.tensor([0] + new), 0)
        pos = torch.cat([torch.arange(h - n, h) for n, h in zip(new, held)] + [torch.zeros(2, dtype=torch.int64)])
        if step == 4:
            pos = pos * 3 + 11  # positions of their own
        out_q = torch.full((total, Hq, D), 7.0, dtype=dtype, device="cuda")
        single = new == [1] * S
        args = (None, 1) if single else (_i32(cu.tolist()), max(new))
        if single:
            q, k, v, out_q, pos = (x[:S] for x in (q, k, v, out_q, pos))
        got = ta.kv_cache_append(cache, k.cuda(), v.cuda(), _i32(table.tolist()), _i32(held), *args, rotary=rot,
                                 q=q.cuda(), out_q=out_q, positions=_i32(pos.tolist()) if step == 4 else None)
        torch.cuda.synchronize()
        assert ta.get_status() == 0 and got is out_q
        n = sum(new)
        want_q, want_k = ta.rotary_embedding(q.cuda(), k.cuda(), _i32(pos.tolist()), rot)
        assert torch.equal(got[:n], want_q[:n]) and bool((got[n:] == 7.0).all())
        k64, _ = _turn64(k, pos, rot)
        for s in range(S):
            a, b = int(cu[s]), int(cu[s + 1])
            if a < b:
                rows = k64 if codes else want_k.double().cpu()
                model["k"].append(table[s], held[s], rows[a:b], codes)
                model["v"].append(table[s], held[s], v[a:b].double(), codes)
    for x in "kv":
        c = getattr(cache, x)
        values = c.float().double().cpu()
        seen = torch.zeros(pages, P, dtype=torch.bool)
        for (page, off), row in model[x].rows.items():
            seen[page, off] = True
            have = values[page, :, off]
            if not codes:
                assert torch.equal(have, row)
                continue
            sc = torch.tensor([model[x].scale[(page, h)] for h in range(Hk)], dtype=torch.float64)[:, None]
            assert torch.equal(getattr(cache, x + "_scale")[page].double().cpu(), sc[:, 0])
            mag = 2 * rot.attention_factor * row.abs().amax() if x == "k" else 0.0
            err, tol = (have * sc - row).abs(), 2.0 ** -4 * row.abs() + 3 * 2.0 ** -10 * sc + mag * 2.0 ** -21
            assert bool((err <= tol).all()), float((err - tol).max())
        raw = c.view(torch.uint8 if codes else cdtype).cpu()
        assert torch.equal(raw.transpose(1, 2)[~seen], untouched[x].cpu().transpose(1, 2)[~seen])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_codes_are_the_nearest(dtype):
    """Every kind of value in one page without a rotation: bit for bit the nearest code, NaN in its own place."""
    import masked_attention_tri_gb300 as ta
    D, P, Hk = 64, 32, 3
    g = torch.Generator().manual_seed(4)
    x = torch.randn(P, Hk, D, generator=g) * torch.exp2(torch.randint(-14, 1, (P, Hk, D), generator=g).float())
    x[:, 1] = 0.0
    x[5, 0, 3], x[6, 0, 4], x[7, 0, 5], x[8, 0, 6] = math.inf, -math.inf, math.nan, 448.0 / 256
    x[:, 2, 0] = 448 * 2.0 ** -20  # the border of a scale: 448 itself
    x[:, 2, 1:] *= 2.0 ** -26
    x = x.to(dtype)
    cache = _filled(2, Hk, P, D, torch.float8_e4m3fn, "")
    r = ta.kv_cache_append(cache, x.cuda(), x.cuda(), _i32([[1]]), _i32([P]), _i32([0, P]), P)
    torch.cuda.synchronize()
    assert r is None and ta.get_status() == 0
    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        for h in range(Hk):
            y = x[:, h].float()
            fin = torch.where(torch.isfinite(y), y, torch.zeros(()))
            sc = _scale64(float(fin.abs().max()))
            assert float(s[1, h]) == sc
            want = torch.where(torch.isfinite(y), y / sc, torch.full((), math.nan)).to(torch.float8_e4m3fn).float()
            assert torch.equal(torch.nan_to_num(c[1, h].float().cpu(), nan=-999.0), torch.nan_to_num(want, nan=-999.0))
        assert bool((c.view(torch.uint8)[0] == 0x35).all()) and bool((s[0] == 0.5).all())


@pytest.mark.gpu
def test_scales_at_the_ends_and_of_another_kind():
    import masked_attention_tri_gb300 as ta
    cache = _filled(1, 1, 16, 16, torch.float8_e4m3fn, "")
    big = torch.full((1, 1, 16), 3e38, device="cuda")
    small = torch.full((1, 1, 16), 1e-38, device="cuda")
    ta.kv_cache_append(cache, big, small, _i32([[0]]), _i32([1]))
    assert float(cache.k_scale[0, 0]) == 2.0 ** 56 and float(cache.v_scale[0, 0]) == 2.0 ** -56
    assert bool((cache.k[0, 0, 0].float() == 448).all()) and bool((cache.v[0, 0, 0].float() == 0).all())
    # a scale that is no power of two (a cache filled by other means) is kept while it covers the rows
    cache.k_scale.fill_(0.3)
    ta.kv_cache_append(cache, torch.full((1, 1, 16), 3.0, device="cuda"), small, _i32([[0]]), _i32([2]))
    assert abs(float(cache.k_scale[0, 0]) - 0.3) < 1e-7 and bool((cache.k[0, 0, 1].float() == 10).all())


@pytest.mark.gpu
def test_broken_contracts_are_skipped():
    import masked_attention_tri_gb300 as ta
    cache = _filled(3, 2, 16, 32, torch.float16, "")
    before = cache.k.clone()
    k = torch.ones(4, 2, 32, dtype=torch.float16, device="cuda")
    run = lambda table, held, cu, most: ta.kv_cache_append(cache, k, k, _i32(table), _i32(held), _i32(cu), most)  # noqa: E731
    for table, held, cu, most in (([[3]], [4], [0, 4], 4), ([[-1]], [4], [0, 4], 4),   # pages out of range
                                  ([[0]], [17], [0, 4], 4), ([[0]], [3], [0, 4], 4),   # beyond the table; fewer than new
                                  ([[0]], [-2147483648], [0, 4], 4),
                                  ([[0]], [4], [0, 4], 3), ([[0]], [4], [0, 5], 5),    # beyond max_seqlen; beyond total
                                  ([[0]], [4], [-1, 3], 4), ([[0]], [4], [4, 0], 4)):
        run(table, held, cu, most)
        assert ta.get_status() == abi.TA_ERR_DEVICE and ta.get_status() == 0
        assert torch.equal(cache.k, before)
    # a broken sequence beside a sound one
    run([[7], [2]], [2, 2], [0, 2, 4], 2)
    assert ta.get_status() == abi.TA_ERR_DEVICE
    assert bool((cache.k[2, :, :2] == 1).all()) and torch.equal(cache.k[:2], before[:2])


@pytest.mark.gpu
def test_more_jobs_than_a_grid_has():
    """16381 heads (a prime) of whole pages of 1024 rows: refused, nothing written; of single rows: written."""
    import masked_attention_tri_gb300 as ta
    Hk = 16381
    cache = ta.PagedKVCache(*(torch.zeros(1, Hk, 1024, 8, dtype=torch.float16, device="cuda") for _ in range(2)))
    k = torch.ones(1, Hk, 8, dtype=torch.float16, device="cuda")
    with pytest.raises(NotImplementedError):
        ta.kv_cache_append(cache, k, k, _i32([[0]]), _i32([1]), _i32([0, 1]), 1024)
    assert not bool(cache.k.any())
    ta.kv_cache_append(cache, k, k, _i32([[0]]), _i32([1]))
    assert bool((cache.k[0, :, 0] == 1).all()) and not bool(cache.v[0, :, 1:].any())
    assert ta.get_status() == 0


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    """The last page of a cache of more than 2^31 elements."""
    import masked_attention_tri_gb300 as ta
    pages, Hk, P, D = 8200, 8, 128, 256
    assert pages * Hk * P * D > 2 ** 31
    cache = ta.PagedKVCache.empty(pages, Hk, P, D, torch.float8_e4m3fn)
    k = torch.randn(1, Hk, D, device="cuda").bfloat16()
    ta.kv_cache_append(cache, k, -k, _i32([[0, pages - 1]]), _i32([P + 1]))
    for c, s, x in ((cache.k, cache.k_scale, k), (cache.v, cache.v_scale, -k)):
        got = c[pages - 1, :, 0].float() * s[pages - 1][:, None]
        err, tol = (got - x[0].float()).abs(), 2.0 ** -4 * x[0].float().abs() + 2.0 ** -10 * s[pages - 1][:, None]
        assert bool((err <= tol).all())


@pytest.mark.gpu
def test_replayed_and_on_another_stream():
    """A captured single-token append, replayed with new rows and lengths, against eager calls."""
    import masked_attention_tri_gb300 as ta
    S, Hk, D, P, MP = 5, 2, 64, 16, 3
    rot = ta.Rotary(D, device="cuda")
    table = torch.randperm(S * MP, generator=torch.Generator().manual_seed(0)).view(S, MP).to(torch.int32).cuda()
    one, two = (_filled(S * MP, Hk, P, D, torch.float8_e4m3fn, "") for _ in range(2))
    k, v, q = (torch.randn(S, h, D, device="cuda").bfloat16() for h in (Hk, Hk, 4))
    held = _i32([1, 16, 17, 33, 48])
    with torch.cuda.stream(torch.cuda.Stream()):
        ta.kv_cache_append(one, k, v, table, held, rotary=rot, q=q)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = ta.kv_cache_append(one, k, v, table, held, rotary=rot, q=q)
    ta.kv_cache_append(two, k, v, table, held, rotary=rot, q=q)
    for step in range(3):
        for t in (k, v, q):
            t.copy_(torch.randn_like(t) * 10 ** step)
        held.copy_(_i32([2 + step, 17 + step, 18 + step, 34 + step, 47]))
        graph.replay()
        want = ta.kv_cache_append(two, k, v, table, held, rotary=rot, q=q)
        assert torch.equal(out, want)
    for a, b in ((one.k, two.k), (one.v, two.v)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(one.k_scale, two.k_scale) and ta.get_status() == 0
