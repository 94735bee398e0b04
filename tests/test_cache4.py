"""The 4-bit paged cache: written, read back and attended to; reading the other caches back; refusals on the CPU.

Codes and scales.  Without a rotation an appended element's arithmetic is exact up to two correctly rounded fp32 divisions
(by 7, by the scale) of numbers whose quotients of 16-bit inputs are exact where they lie on a border: codes and scales have
to be the definition's, bit for bit (the definition below divides in fp64 and, for fp32 inputs, passes over elements within
2^-22 of a border).  With a rotation a key is off by (|a| + |b|) m 2^-21 before it is coded (test_rotary.py), so a
value read back is off by at most that and the coding's own error: half a step of n, s f / 2; an element of the largest magnitude
lies at most 7 (1 + 2^-4) steps out, where n = 7 is off by 7 2^-4; and s itself moves with the group's largest element.  The test
takes |value - x| <= (0.5 + 2^-5) s f + 2^-21 m (|a| + |b|) with the kernel's own s, which has to be within e4m3's half step
(2^-4, or 2^-10 below 2^-6) of max |x| / 7 f.

Attention: as in test_paged_attention.py, with the weights in fp16, and queries of 16 bits as fp16 numbers scaled so that the
row's largest is in [1, 2): off by 2^-25 of that magnitude at most, which moves a logit by scale 2^-24 max|q| sum |k|.
"""
import math

import pytest
import torch

from masked_attention_tri_gb300 import abi, build
from test_rotary import _turn64

A = 0x10000
BF, F16, F32, F8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


# ---------------------------------------------------------------------------- CPU

def _c4(**kw):
    args = dict(k=A, v=A, k_scale=A, v_scale=A, k_factor=None, v_factor=None, num_pages=4, page_size=64)
    args.update(kw)
    strides = args.pop("strides", (0,) * 8)
    c = abi.Cache4(**args)
    for i, s in enumerate(strides):
        c.strides[i] = s
    return c


def _append(**kw):
    args = dict(q=A, k=A, v=A, dtype=abi.TA_BF16, cu_seqlens=A, kv_lengths=A, page_table=A, num_seqs=2, total=8,
                max_seqlen=4, Hq=4, Hk=2, D=64, q_row_stride=0, k_row_stride=0, v_row_stride=0, q_out_row_stride=0,
                positions=0, num_axes=1, pair_axes=0, turns=A, rotary_dim=64, interleaved=0, mscale=1.0, cache=_c4(),
                max_pages=2, q_out=A, stream=0)
    args.update(kw)
    return abi.tri_attn_kv_append4(**args)


def _paged(**kw):
    args = dict(q=A, dtype=abi.TA_BF16, cu_seqlens_q=A, kv_lengths=A, page_table=A, num_seqs=2, total_q=8, max_seqlen_q=4,
                Hq=4, Hk=2, D=64, q_row_stride=0, scale=0.125, window=0, sinks=0, cache=_c4(), max_pages=2, out=A, lse=A,
                workspace=A, workspace_bytes=1 << 30, stream=0)
    args.update(kw)
    return abi.tri_attn_paged4_fwd(**args)


def _read(**kw):
    args = dict(cu_seqlens=A, kv_lengths=A, page_table=A, num_seqs=2, total=8, max_seqlen=4, Hk=2, D=64, cache=_c4(),
                max_pages=2, k_out=A, v_out=A, dtype=abi.TA_BF16, k_row_stride=0, v_row_stride=0, stream=0)
    args.update(kw)
    return abi.tri_attn_kv_read4(**args)


CACHES = [(dict(k=None), ValueError), (dict(v_scale=None), ValueError), (dict(k=A + 8), ValueError),
          (dict(k_scale=A + 8), ValueError), (dict(k_factor=A + 2), ValueError), (dict(num_pages=0), ValueError),
          (dict(page_size=0), ValueError), (dict(page_size=24), NotImplementedError),
          (dict(page_size=2048), NotImplementedError), (dict(page_size=8), NotImplementedError),
          (dict(strides=(4096, 2048 - 16) * 2 + (512, 256) * 2), ValueError),
          (dict(strides=(4096, 2056) * 2 + (512, 256) * 2), NotImplementedError)]


@pytest.mark.parametrize("kw,exc", CACHES)
def test_caches_refused(kw, exc):
    for call in (_append, _paged, _read):
        with pytest.raises(exc):
            call(cache=_c4(**kw))


@pytest.mark.parametrize("kw,exc", [
    (dict(cache=None), ValueError), (dict(max_pages=0), ValueError), (dict(num_seqs=0), ValueError),
    (dict(kv_lengths=0), ValueError), (dict(page_table=0), ValueError), (dict(dtype=abi.TA_INT4), ValueError),
    (dict(dtype=abi.TA_E4M3), ValueError), (dict(Hk=0), ValueError), (dict(D=80, rotary_dim=64), NotImplementedError),
    (dict(D=288), NotImplementedError)])
def test_calls_refused(kw, exc):
    for call in (_append, _paged, _read):
        with pytest.raises(exc):
            call(**({k: v for k, v in kw.items() if k != "rotary_dim"} if call is not _append else kw))


@pytest.mark.parametrize("call,kw,exc", [
    (_append, dict(k=0), ValueError), (_append, dict(q_out=0), ValueError), (_append, dict(rotary_dim=48), NotImplementedError),
    (_append, dict(num_axes=2), ValueError), (_append, dict(pair_axes=A, num_axes=0), ValueError),
    (_append, dict(pair_axes=A + 2, num_axes=2), ValueError),
    (_append, dict(pair_axes=A, num_axes=2, turns=0, rotary_dim=0, q=0, q_out=0, Hq=0), ValueError),
    (_read, dict(k_out=0), ValueError), (_read, dict(v_out=A + 8), ValueError), (_read, dict(total=-1), ValueError),
    (_read, dict(cu_seqlens=0), ValueError), (_read, dict(k_row_stride=64), ValueError),
    (_read, dict(k_row_stride=132), NotImplementedError),
    (_paged, dict(workspace_bytes=16), ValueError), (_paged, dict(Hk=3), ValueError), (_paged, dict(window=-1), ValueError)])
def test_each_refused(call, kw, exc):
    with pytest.raises(exc):
        call(**kw)


@pytest.mark.parametrize("kw,exc", [
    (dict(k_cache=0), ValueError), (dict(cache_dtype=abi.TA_F16), NotImplementedError), (dict(k_scale=A), ValueError),
    (dict(cache_dtype=abi.TA_E4M3), ValueError), (dict(cache_dtype=abi.TA_INT4), ValueError),
    (dict(page_size=24), NotImplementedError), (dict(v_out=0), ValueError)])
def test_read_of_other_caches_refused(kw, exc):
    args = dict(cu_seqlens=A, kv_lengths=A, page_table=A, num_seqs=2, total=8, max_seqlen=4, Hk=2, D=64, k_cache=A, v_cache=A,
                cache_dtype=abi.TA_BF16, k_scale=0, v_scale=0, num_pages=4, page_size=64, max_pages=2, k_strides=None,
                v_strides=None, k_out=A, v_out=A, dtype=abi.TA_BF16, k_row_stride=0, v_row_stride=0, stream=0)
    args.update(kw)
    with pytest.raises(exc):
        abi.tri_attn_kv_read(**args)


def test_four_bits_belong_to_their_own_calls():
    with pytest.raises(ValueError):
        abi.tri_attn_paged_fwd(q=A, dtype=abi.TA_BF16, cu_seqlens_q=A, kv_lengths=A, page_table=A, num_seqs=2, total_q=8,
                               max_seqlen_q=4, Hq=4, Hk=2, D=64, q_row_stride=0, scale=0.125, window=0, sinks=0, k_cache=A,
                               v_cache=A, cache_dtype=abi.TA_INT4, k_scale=0, v_scale=0, num_pages=4, page_size=64,
                               max_pages=2, k_strides=None, v_strides=None, out=A, lse=A, workspace=A,
                               workspace_bytes=1 << 30, stream=0)


def test_nothing_to_do():
    _append(total=0)
    _append(max_seqlen=0)
    _read(total=0)
    _read(max_seqlen=0)
    _paged(total_q=0)


def test_handle_refusals():
    import masked_attention_tri_gb300 as ta
    k = torch.zeros(3, 2, 16, 32, dtype=torch.uint8)
    s = torch.zeros(3, 2, 16, 4, dtype=torch.uint8).view(F8)
    c = ta.PagedKVCache4(k, k.clone(), s, s.clone(), torch.ones(2))
    assert (c.num_pages, c.heads, c.page_size, c.head_dim) == (3, 2, 16, 64)
    for bad in ((k[0], k, s, s), (k, k[:2], s, s), (k, k, s[:, :1], s), (k, k, s, s, torch.ones(3)),
                (k.transpose(2, 3), k.transpose(2, 3), s, s), (k[..., :8], k[..., :8], s[..., :1], s[..., :1])):
        with pytest.raises(ValueError):
            ta.PagedKVCache4(*bad)
    with pytest.raises(TypeError):
        ta.PagedKVCache4(k.int(), k.int(), s, s)
    with pytest.raises(TypeError):
        ta.PagedKVCache4(k, k, s.float(), s.float())
    i32 = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):  # on the CPU
        ta.kv_cache_read(c, i32[None], i32)
    with pytest.raises(TypeError):
        ta.kv_cache_read(k, i32[None], i32)


# ---------------------------------------------------------------------------- the definition

E4M3 = torch.arange(127, dtype=torch.uint8).view(F8).double()


def _define(x, factor):
    """(n, scale, sure) of rows x (..., D): the whole numbers, the scales, and where neither is near a border."""
    y = (x.double() / factor).unflatten(-1, (-1, 16))
    a = (y.abs().amax(-1) / 7).clamp(2.0 ** -9, 448.0)
    table = E4M3.to(x.device)
    i = torch.searchsorted(table, a.contiguous()).clamp(1, 126)
    lo, hi = table[i - 1], table[i]
    up = (a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 0))
    s = torch.where(up, hi, lo)
    z = y / s[..., None]
    n = torch.round(z).clamp(-7, 7)
    exact = x.dtype != F32
    mid = ((a - (lo + hi) / 2).abs() > 2.0 ** -22 * a) | exact
    sure = (((z - z.floor() - 0.5).abs() > 2.0 ** -22 * 8) | exact) & mid[..., None]
    return n.flatten(-2), s, sure.flatten(-2)


def _unpack(b):
    return torch.stack((b & 15, b >> 4), -1).flatten(-2).double() - 8


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cu(n):
    return [0] + [sum(n[:i + 1]) for i in range(len(n))]


def _cache(pages, Hk, P, D, seed=0, strided=False, factors=True, poison=False):
    """A cache full of random codes (or of NaN scales), so that what is left alone can be told."""
    import masked_attention_tri_gb300 as ta
    g = torch.Generator(device="cuda").manual_seed(seed)
    if strided:
        kv = torch.randint(0, 256, (pages, 2, Hk, P, D // 2), generator=g, device="cuda", dtype=torch.uint8)
        k, v = kv[:, 0], kv[:, 1]
        sc = torch.empty(pages, Hk, 2, P, D // 16, dtype=torch.uint8, device="cuda")
        ks, vs = sc[:, :, 0], sc[:, :, 1]
    else:
        k, v = (torch.randint(0, 256, (pages, Hk, P, D // 2), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2))
        ks, vs = (torch.empty(pages, Hk, P, D // 16, dtype=torch.uint8, device="cuda") for _ in range(2))
    for s in (ks, vs):
        s.copy_(torch.full(s.shape, 0x7f, dtype=torch.uint8, device="cuda") if poison else
                (torch.rand(s.shape, generator=g, device="cuda") * 3 + 0.01).to(F8).view(torch.uint8))
    f = [torch.exp2(torch.randint(-3, 4, (Hk,), generator=g, device="cuda").float()) if factors else None for _ in range(2)]
    return ta.PagedKVCache4(k, v, ks.view(F8), vs.view(F8), *f)


def _tables(helds, P, spare=1, seed=0):
    g = torch.Generator().manual_seed(seed)
    need = [-(-h // P) for h in helds]
    order = torch.randperm(sum(need) + spare, generator=g).tolist()
    MP = max(need + [1]) + 1
    rows = []
    for n in need:
        rows.append([order.pop() for _ in range(n)] + [-3] * (MP - n))
    return _i32(rows), sum(need) + spare


def _slots_of(table, news, helds, P):
    page, off = [], []
    for i, (n, h) in enumerate(zip(news, helds)):
        for t in range(h - n, h):
            page.append(int(table[i, t // P]))
            off.append(t % P)
    return torch.tensor(page, device="cuda", dtype=torch.long), torch.tensor(off, device="cuda", dtype=torch.long)


# ---------------------------------------------------------------------------- GPU

CASES = [
    # new tokens, slots after, Hk, D, page, dtype
    ([1], [1], 1, 32, 16, BF),
    ([1, 1, 1], [1, 64, 65], 8, 128, 64, BF),
    ([3, 0, 40, 17], [3, 9, 100, 130], 2, 64, 16, F16),
    ([200, 1], [200, 33], 4, 128, 64, BF),
    ([70], [1000], 3, 96, 32, F32),
    ([33, 5], [33, 300], 2, 256, 128, BF),
    ([1025], [1025], 1, 160, 1024, F16),
    ([257], [300], 5, 224, 16, F32),
]


@pytest.mark.gpu
@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("news,helds,Hk,D,P,dtype", CASES)
def test_append(news, helds, Hk, D, P, dtype, strided):
    import masked_attention_tri_gb300 as ta
    table, pages = _tables(helds, P)
    cache = _cache(pages, Hk, P, D, strided=strided)
    before = [t.clone() for t in (cache.k, cache.v, cache.k_scale.view(torch.uint8), cache.v_scale.view(torch.uint8))]
    g = torch.Generator(device="cuda").manual_seed(1)
    total = sum(news)
    x = [(torch.randn(total + 3, Hk, D, generator=g, device="cuda") *
          torch.exp2(torch.randint(-12, 10, (total + 3, Hk, D // 16), generator=g, device="cuda").float()).repeat_interleave(16, -1)).to(dtype)
         for _ in range(2)]
    x[0][0, 0, :16] = 0
    cu = _i32(_cu(news))
    ta.kv_cache_append(cache, x[0], x[1], table, _i32(helds), cu, max(news))
    assert ta.get_status() == 0
    page, off = _slots_of(table, news, helds, P)
    for i, (codes, scale, f) in enumerate(((cache.k, cache.k_scale, cache.k_factor), (cache.v, cache.v_scale, cache.v_factor))):
        n, s, sure = _define(x[i][:total], f.double()[:, None])
        got_s = scale.view(torch.uint8)[page, :, off].view(F8).double()
        got_n = _unpack(codes[page, :, off])
        fine = sure.unflatten(-1, (-1, 16)).all(-1) if dtype == F32 else torch.ones_like(s, dtype=torch.bool)
        assert float(fine.double().mean()) > 0.99
        assert bool(((got_s == s) | ~fine).all())
        assert bool(((got_n == n) | ~sure).all())
        mask = torch.ones(codes.shape[:3], dtype=torch.bool, device="cuda").transpose(1, 2)
        mask[page, off] = False
        for now, then in ((codes, before[i]), (scale.view(torch.uint8), before[2 + i])):
            assert bool((now.transpose(1, 2)[mask] == then.transpose(1, 2)[mask]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("axes", [False, True])
@pytest.mark.parametrize("dtype,D,dim,inter", [(BF, 128, 128, False), (F16, 128, 64, True), (F32, 64, 64, False),
                                               (F32, 96, 32, True), (BF, 96, 32, False)])
def test_append_with_rotation(dtype, D, dim, inter, axes):
    import masked_attention_tri_gb300 as ta
    news, helds, Hk, Hq, P = [5, 40, 1], [20, 40, 64], 2, 4, 32
    table, pages = _tables(helds, P)
    cache = _cache(pages, Hk, P, D)
    rot = ta.Rotary(dim, interleaved=inter, device="cuda", sections=(dim // 2 - 5, 5) if axes else None)
    g = torch.Generator(device="cuda").manual_seed(2)
    total = sum(news)
    q, k, v = (torch.randn(total, h, D, generator=g, device="cuda").to(dtype) for h in (Hq, Hk, Hk))
    pos = torch.randint(0, 5000, (2, total), generator=g, device="cuda", dtype=torch.int32) if axes else None
    cu = _i32(_cu(news))
    got_q = ta.kv_cache_append(cache, k, v, table, _i32(helds), cu, max(news), rotary=rot, positions=pos, q=q)
    slots = torch.cat([torch.arange(h - n, h, dtype=torch.int32) for n, h in zip(news, helds)]).cuda()
    assert bool((got_q == ta.rotary_embedding(q, None, pos if axes else slots, rot)).all())
    if axes:
        import test_rotary_axes
        want, mag = test_rotary_axes._turn64(k, pos, rot)
    else:
        want, mag = _turn64(k, slots, rot)
    want, mag = want.cuda(), mag.cuda()
    back = ta.kv_cache_read(cache, table, _i32(helds), cu, max(news), total, dtype=F32)
    page, off = _slots_of(table, news, helds, P)
    for x, m, y, scale, f in ((want, mag, back[0], cache.k_scale, cache.k_factor), (v.double(), 0 * mag, back[1], cache.v_scale, cache.v_factor)):
        s = scale.view(torch.uint8)[page, :, off].view(F8).double()
        most = x.unflatten(-1, (-1, 16)).abs().amax(-1) / 7 / f.double()[:, None]
        slack = (m.unflatten(-1, (-1, 16)).amax(-1) * 2.0 ** -21) / 7 / f.double()[:, None]
        assert bool(((s - most).abs() <= 2.0 ** -4 * most + 2.0 ** -10 + slack).all())
        step = (s * f.double()[:, None]).repeat_interleave(16, -1)
        assert bool(((y.double() - x).abs() <= (0.5 + 2.0 ** -5) * step + m * 2.0 ** -21).all())
    # without positions every axis is the slot
    if axes:
        again = _cache(pages, Hk, P, D)
        q2 = ta.kv_cache_append(again, k, v, table, _i32(helds), cu, max(news), rotary=rot, q=q)
        assert bool((q2 == ta.rotary_embedding(q, None, slots.expand(2, -1).contiguous(), rot)).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32, F8])
def test_append_of_axes_to_other_caches(dtype):
    """The rows that go into a 16-bit, fp32 or 8-bit cache with an axis for each pair are those of rotary_embedding."""
    import masked_attention_tri_gb300 as ta
    rows = BF if dtype == F8 else dtype
    helds = [70, 5]
    table, pages = _tables(helds, 32)
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v, q = (torch.randn(75, h, 64, generator=g, device="cuda").to(rows) for h in (2, 2, 4))
    pos = torch.randint(0, 900, (3, 75), generator=g, device="cuda", dtype=torch.int32)
    rot = ta.Rotary(64, sections=(10, 11, 11), section_layout="interleaved", device="cuda")
    caches = [ta.PagedKVCache.empty(pages, 2, 32, 64, dtype) for _ in range(2)]
    for c in caches:
        for t in (c.k, c.v):
            t.view(torch.uint8).zero_()
    lens, cu = _i32(helds), _i32(_cu(helds))
    turned, kt = ta.rotary_embedding(q, k, pos, rot)
    got = ta.kv_cache_append(caches[0], k, v, table, lens, cu, 70, rotary=rot, positions=pos, q=q)
    assert bool((got == turned).all())
    if dtype == F8:  # (codes of the rows before their rounding to 16 bits: half a step of either apart at most)
        y = ta.kv_cache_read(caches[0], table, lens, cu, 70, 75, dtype=F32)[0].double()
        assert bool(((y - kt.double()).abs() <= kt.double().abs() * (2.0 ** -4 + 2.0 ** -8) + 2.0 ** -10 * caches[0].k_scale.max()).all())
    else:
        ta.kv_cache_append(caches[1], kt, v, table, lens, cu, 70)
        used = table[table >= 0].long()
        assert bool((caches[0].k[used] == caches[1].k[used]).all())


@pytest.mark.gpu
def test_infinities_and_nan():
    import masked_attention_tri_gb300 as ta
    table, pages = _tables([3], 16)
    cache = _cache(pages, 1, 16, 64)
    k = torch.ones(3, 1, 64, dtype=BF, device="cuda")
    k[0, 0, 5], k[1, 0, 20], k[2, 0, 63] = math.inf, math.nan, -math.inf
    ta.kv_cache_append(cache, k, torch.ones_like(k) * 3e38, table, _i32([3]), _i32([0, 3]), 3)
    y, v = ta.kv_cache_read(cache, table, _i32([3]), _i32([0, 3]), 3, 3)
    bad = torch.zeros(3, 1, 4, dtype=torch.bool, device="cuda")
    bad[0, 0, 0] = bad[1, 0, 1] = bad[2, 0, 3] = True
    assert bool((torch.isnan(y) == bad.repeat_interleave(16, -1)).all())
    assert bool((v == 3136.0 * cache.v_factor).all())  # beyond the scale's range: its largest number


@pytest.mark.gpu
@pytest.mark.parametrize("cdtype,dtype", [(None, BF), (None, F16), (None, F32), (F8, BF), (F8, F16), (F8, F32), (BF, BF), (F16, F16), (F32, F32)])
@pytest.mark.parametrize("news,helds,Hk,D,P", [c[:5] for c in CASES])
def test_read(news, helds, Hk, D, P, cdtype, dtype):
    import masked_attention_tri_gb300 as ta
    table, pages = _tables(helds, P)
    total = sum(news)
    page, off = _slots_of(table, news, helds, P)
    g = torch.Generator(device="cuda").manual_seed(4)
    if cdtype is None:
        cache = _cache(pages, Hk, P, D, strided=True)
        want = [(_unpack(c[page, :, off]).unflatten(-1, (-1, 16)) * s.view(torch.uint8)[page, :, off].view(F8).double()[..., None]).flatten(-2) * f.double()[:, None]
                for c, s, f in ((cache.k, cache.k_scale, cache.k_factor), (cache.v, cache.v_scale, cache.v_factor))]
    else:
        x = [torch.randn(pages, Hk, P, D, generator=g, device="cuda").to(cdtype) for _ in range(2)]
        sc = [torch.exp2(torch.randint(-9, 9, (pages, Hk), generator=g, device="cuda").float()) for _ in range(2)] if cdtype == F8 else [None, None]
        cache = ta.PagedKVCache(*x, *sc)
        want = []
        for t, s in zip(x, sc):
            y = (t.view(torch.uint8).double() if False else t.to(F32).double())[page, :, off]
            want.append(y if s is None else y * s.double()[page][..., None])
    outs = [torch.full((total + 2, Hk + 1, D), 9.0, dtype=dtype, device="cuda") for _ in range(2)]
    views = [o[:, :Hk] for o in outs]
    k, v = ta.kv_cache_read(cache, table, _i32(helds), _i32(_cu(news)), max(news), out_k=views[0], out_v=views[1])
    assert ta.get_status() == 0
    for o, w in zip(outs, want):  # (one rounding of a product of at most 8 significant bits, or 4 and a power of two)
        assert bool((o[:total, :Hk] == w.to(dtype)).all())
        assert bool((o[total:] == 9).all()) and bool((o[:, Hk] == 9).all())
    k2, v2 = ta.kv_cache_read(cache, table, _i32(helds), _i32(_cu(news)), max(news), total, dtype=dtype)
    assert bool((k2 == k[:total]).all()) and bool((v2 == v[:total]).all())


@pytest.mark.gpu
def test_read_of_a_prefix_and_of_single_rows():
    import masked_attention_tri_gb300 as ta
    helds = [100, 40, 7]
    table, pages = _tables(helds, 16)
    cache = _cache(pages, 2, 16, 64)
    k, v = ta.kv_cache_read(cache, table, _i32(helds), _i32(_cu(helds)), 100, sum(helds))
    pre = [60, 0, 7]
    k1, v1 = ta.kv_cache_read(cache, table, _i32(pre), _i32(_cu(pre)), 60, sum(pre))
    assert bool((k1 == torch.cat((k[:60], k[140:147]))).all()) and bool((v1 == torch.cat((v[:60], v[140:147]))).all())
    k1, v1 = ta.kv_cache_read(cache, table, _i32(helds))
    assert bool((k1 == k[[99, 139, 146]]).all()) and bool((v1 == v[[99, 139, 146]]).all())


@pytest.mark.gpu
def test_broken_sequences_and_pages_are_skipped():
    import masked_attention_tri_gb300 as ta
    helds = [20, 20]
    table, pages = _tables(helds, 16)
    cache = _cache(pages, 2, 16, 64)
    k = torch.randn(40, 2, 64, device="cuda").to(BF)
    codes = cache.k.clone()
    ta.get_status()
    for cu, lens, tab in (([0, 30, 40], [20, 20], table), ([0, 20, 50], [20, 20], table), ([0, 20, 40], [20, 99], table),
                          ([0, 20, 40], [20, 20], _i32([[pages, -1, 0], [pages + 5, 1 << 30, 0]]))):
        kv = _i32(lens)
        ta.kv_cache_append(cache, k, k, tab, kv, _i32(cu), 20)
        assert ta.get_status() == abi.TA_ERR_DEVICE
        ta.kv_cache_read(cache, tab, kv, _i32(cu), 20, 40)
        assert ta.get_status() == abi.TA_ERR_DEVICE
    out = ta.paged_attention(torch.ones(2, 4, 64, dtype=BF, device="cuda"), cache, _i32([[pages, -1, 0], [pages + 5, 1 << 30, 0]]), _i32(helds))
    assert ta.get_status() == abi.TA_ERR_DEVICE and bool((out == 0).all())
    assert codes.shape == cache.k.shape


class Problem:
    """Sequences over a 4-bit cache; scales of slots that no row sees are NaN, unneeded table entries out of range."""

    def __init__(self, news, helds, Hq, Hk, D, P, dtype, window=None, sinks=0, spread=1.0, seed=0, strided=False):
        self.news, self.helds, self.window, self.sinks = news, helds, window, sinks
        self.table, pages = _tables(helds, P, seed=seed)
        self.cache = _cache(pages, Hk, P, D, seed=seed, strided=strided, poison=True)
        g = torch.Generator(device="cuda").manual_seed(seed + 9)
        self.q = (torch.randn(sum(news), Hq, D, generator=g, device="cuda") * spread).to(dtype)
        self.see = []
        for i, (n, h) in enumerate(zip(news, helds)):
            pos, j = torch.arange(h - n, h, device="cuda")[:, None], torch.arange(h, device="cuda")
            see = j <= pos
            if window:
                see = see & ((pos - j < window) | (j < sinks))
            self.see.append(see)
            at = torch.nonzero(see.any(0)).flatten()
            page, off = self.table[i].long()[at // P], at % P
            for s in (self.cache.k_scale, self.cache.v_scale):
                sc = torch.exp2(torch.rand(len(at), Hk, D // 16, generator=g, device="cuda") * 6 - 5).to(F8)
                s.view(torch.uint8)[page, :, off] = sc.view(torch.uint8)
            for lp in range(-(-h // P)):
                if not bool(see.any(0)[lp * P:(lp + 1) * P].any()):
                    self.table[i, lp] = -9
        self.P = P

    def rows(self, i, kind):
        codes, scale, f = ((self.cache.k, self.cache.k_scale, self.cache.k_factor), (self.cache.v, self.cache.v_scale, self.cache.v_factor))[kind]
        h = self.helds[i]
        j = torch.arange(h, device="cuda")
        page, off = self.table[i].long()[j // self.P].clamp(min=0), j % self.P
        y = _unpack(codes[page, :, off]).unflatten(-1, (-1, 16)) * scale.view(torch.uint8)[page, :, off].view(F8).double()[..., None]
        return (y.flatten(-2) * f.double()[:, None]).nan_to_num(0.0)  # (h, Hk, D)

    def check(self, scale=None):
        import masked_attention_tri_gb300 as ta
        q, c = self.q, self.cache
        s = float(torch.tensor(1 / math.sqrt(q.shape[2]) if scale is None else scale, dtype=torch.float32))
        cu = _i32(_cu(self.news)) if max(self.news) > 1 or 0 in self.news else None
        o, lse = ta.paged_attention(q, c, self.table, _i32(self.helds), cu, max(self.news), scale, window=self.window,
                                    sinks=self.sinks, return_aux=True)
        assert ta.get_status() == 0
        Hq, Hk, D = q.shape[1], c.heads, q.shape[2]
        eps, half = torch.finfo(q.dtype).eps, q.dtype != F32
        t = 0
        for i, (n, h) in enumerate(zip(self.news, self.helds)):
            if not n:
                continue
            K, V = self.rows(i, 0), self.rows(i, 1)
            see = self.see[i]
            for a in range(Hq):
                Q = q[t:t + n, a].double()
                x = s * (Q @ K[:, a // (Hq // Hk)].t())
                E = abs(s) * (Q.abs() @ K[:, a // (Hq // Hk)].abs().t()).masked_fill(~see, 0)
                dx = D * 2.0 ** -23 * E.amax(1) + 2.0 ** -22 * x.masked_fill(~see, 0).abs().amax(1)
                if half:
                    dx = dx + abs(s) * 2.0 ** -24 * Q.abs().amax(1) * K[:, a // (Hq // Hk)].abs().sum(1).masked_fill(~see, 0).amax(1)
                x = x.masked_fill(~see, -math.inf)
                L = torch.logsumexp(x, 1)
                w = (x - L[:, None]).exp()
                Vh = V[:, a // (Hq // Hk)]
                rel = (2.0 ** -11 if half else 2.0 ** -24) + 2 * dx + 2.0 ** -21 + h * 2.0 ** -23
                R = w @ Vh
                tol = eps / 2 * R.abs() + rel[:, None] * (w @ Vh.abs())
                if half:  # fp16's least step: of a weight (relative to the largest), and of an fp16 output
                    tol = tol + 2.0 ** -25 * w.amax(1, keepdim=True) * (see.double() @ Vh.abs())
                if q.dtype == F16:
                    tol = tol + 2.0 ** -25
                err = (o[t:t + n, a].double() - R).abs()
                assert bool((err <= tol).all()), (i, a, float((err - tol).max()))
                e2 = (lse[a, t:t + n].double() - L).abs()
                assert bool((e2 <= dx + 2.0 ** -21 + h * 2.0 ** -24 + 2.0 ** -23 * L.abs()).all()), float(e2.max())
            t += n
        return o


PAGED = [
    # new tokens, slots, Hq, Hk, D, page, dtype, window, sinks
    ([1], [1], 1, 1, 32, 16, BF, None, 0),
    ([1], [1000], 32, 8, 128, 64, BF, None, 0),
    ([1, 1, 1], [15, 16, 17], 4, 2, 64, 16, F16, None, 0),
    ([1, 1], [129, 700], 8, 1, 128, 16, BF, None, 0),
    ([1, 1, 1, 1], [3000, 40, 1, 257], 4, 4, 256, 32, BF, None, 0),
    ([5, 1, 0, 8], [5, 300, 20, 1025], 4, 2, 64, 128, BF, None, 0),
    ([2, 7], [600, 90], 12, 2, 96, 64, F16, None, 0),
    ([1, 3], [900, 2000], 6, 2, 160, 64, BF, None, 0),
    ([1], [5000], 8, 8, 64, 1024, F16, None, 0),
    ([40], [400], 4, 1, 128, 32, BF, None, 0),
    ([1, 4], [3000, 700], 8, 2, 128, 64, BF, 130, 4),
    ([1, 2], [900, 300], 4, 1, 64, 16, F16, 17, 0),
    ([3], [700], 2, 1, 224, 32, BF, 100, 70),
    ([1, 1], [70, 1], 4, 2, 64, 16, F32, None, 0),
    ([3, 1], [130, 999], 6, 1, 128, 64, F32, 50, 3),
    ([1], [400], 3, 3, 256, 32, F32, None, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("news,helds,Hq,Hk,D,P,dtype,window,sinks", PAGED)
def test_attention(news, helds, Hq, Hk, D, P, dtype, window, sinks):
    Problem(news, helds, Hq, Hk, D, P, dtype, window, sinks).check()


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(spread=40.0), dict(spread=1e-4), dict(strided=True), dict(seed=5)])
def test_attention_spread_and_strides(kw):
    Problem([1, 2, 1], [300, 70, 2100], 8, 2, 128, 32, BF, **kw).check()
    Problem([1, 2, 1], [300, 70, 900], 8, 2, 64, 32, F16, **kw).check(scale=-0.3)


@pytest.mark.gpu
def test_attention_of_many_and_of_long_sequences():
    import random
    r = random.Random(1)
    Problem([1] * 300, [r.choice([1, 2, 30, 400]) for _ in range(300)], 4, 2, 64, 16, BF).check()
    Problem([1], [40000], 8, 1, 128, 64, BF).check()


@pytest.mark.gpu
def test_a_row_that_sees_nothing():
    import masked_attention_tri_gb300 as ta
    P = Problem([1, 1], [50, 20], 4, 2, 64, 16, BF)
    o, lse = ta.paged_attention(P.q, P.cache, P.table, _i32([50, 0]), return_aux=True)
    assert bool((o[1] == 0).all()) and bool((lse[:, 1] == -math.inf).all()) and not bool(torch.isnan(o).any())


@pytest.mark.gpu
def test_the_same_every_time_and_captured():
    import masked_attention_tri_gb300 as ta
    P = Problem([1, 1, 1], [5000, 70, 1300], 8, 2, 128, 64, BF)
    lens = _i32(P.helds)
    want = ta.paged_attention(P.q, P.cache, P.table, lens)
    assert all(bool((ta.paged_attention(P.q, P.cache, P.table, lens) == want).all()) for _ in range(3))
    k = torch.randn(3, 2, 128, device="cuda").to(BF)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        ta.kv_cache_append(P.cache, k, k, P.table, lens)
        kk, vv = ta.kv_cache_read(P.cache, P.table, lens)
        o = ta.paged_attention(P.q, P.cache, P.table, lens)
    for _ in range(2):
        k.normal_()
        graph.replay()
        ta.kv_cache_append(P.cache, k, k, P.table, lens)
        assert bool((ta.paged_attention(P.q, P.cache, P.table, lens) == o).all())
        assert bool((ta.kv_cache_read(P.cache, P.table, lens)[0] == kk).all())
    assert ta.get_status() == 0


@pytest.mark.gpu
def test_a_request_from_prompt_to_answer():
    """Positions with three axes, the prompt in two chunks whose prefix is read back, and new tokens: against the same
    computed in fp64 from the rows that the cache holds."""
    import masked_attention_tri_gb300 as ta
    from test_prompt_attention import reference, _within
    Hq, Hk, D, P = 8, 2, 128, 32
    chunks, helds = [[70, 33], [50, 100], [1, 1]], [0, 0]
    final = [121, 134]
    table, pages = _tables(final, P)
    cache = _cache(pages, Hk, P, D, poison=True)
    rot = ta.Rotary(D, sections=(24, 20, 20), device="cuda")
    g = torch.Generator(device="cuda").manual_seed(11)
    for news in chunks:
        helds = [h + n for h, n in zip(helds, news)]
        n = sum(news)
        q, k, v = (torch.randn(n, h, D, generator=g, device="cuda").to(BF) for h in (Hq, Hk, Hk))
        pos = torch.randint(0, 300, (3, n), generator=g, device="cuda", dtype=torch.int32)
        cu, lens = _i32(_cu(news)), _i32(helds)
        q = ta.kv_cache_append(cache, k, v, table, lens, cu, max(news), rotary=rot, positions=pos, q=q)
        cu_k = _i32(_cu(helds))
        kk, vv = ta.kv_cache_read(cache, table, lens, cu_k, max(helds), sum(helds))
        o, lse = ta.prompt_attention(q, kk, vv, cu, cu_k, max(news), max(helds), return_aux=True)
        R, T = reference(q, kk, vv, news, helds, float(torch.tensor(D ** -0.5, dtype=torch.float32)))
        _within(o, R, T, "o")
        # the paged form gives the same: its weights are rounded to fp16 and not to bf16
        o2, lse2 = ta.paged_attention(q, cache, table, lens, cu, max(news), return_aux=True)
        _within(o2, R, T, "o")
        _within(lse2, R, T, "lse")
    assert ta.get_status() == 0
