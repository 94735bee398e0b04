"""Attention over a paged cache at the edges of what its documentation allows."""
import pytest
import torch

from masked_attention_tri_gb300 import abi, build
from test_paged_attention import _call, _i32


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def test_nothing_to_do_needs_no_workspace():
    assert abi.tri_attn_paged_workspace_size(abi.TA_BF16, 0, 4, 2, 64) == 0
    _call(max_seqlen_q=0, workspace=0, workspace_bytes=0)
    _call(total_q=0, workspace=0, workspace_bytes=0)
    with pytest.raises(ValueError):
        _call(workspace=0)


def _cache(pages, Hk, P, D, dtype):
    import masked_attention_tri_gb300 as ta
    k, v = (torch.randn(pages, Hk, P, D, device="cuda").to(dtype) for _ in range(2))
    sc = (torch.ones(pages, Hk, device="cuda"), torch.ones(pages, Hk, device="cuda")) if dtype == torch.float8_e4m3fn else ()
    return ta.PagedKVCache(k, v, *sc)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_no_sequence_has_a_new_token(dtype):
    """max_seqlen_q 0 with rows in q: they lie behind the last sequence and are left as they were."""
    import masked_attention_tri_gb300 as ta
    cache, q = _cache(2, 1, 16, 64, dtype), torch.randn(3, 2, 64, device="cuda").to(dtype)
    out = torch.full_like(q, 7.0)
    r, lse = ta.paged_attention(q, cache, _i32([[0], [1]]), _i32([3, 0]), _i32([0, 0, 0]), 0, out=out, return_aux=True)
    torch.cuda.synchronize()
    assert r is out and bool((out == 7.0).all()) and lse.shape == (2, 3) and ta.get_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,cdtype", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                          (torch.bfloat16, torch.float8_e4m3fn), (torch.float32, torch.float8_e4m3fn)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_logits_far_below_zero(dtype, cdtype, D):
    """Every logit of a row far below zero, and of another far above; the largest alone counts.  The sums behind them,
    2 D mag at most, stay below fp32's 2^128."""
    import masked_attention_tri_gb300 as ta
    n, P = 40, 16
    e4 = cdtype == torch.float8_e4m3fn
    k = torch.full((3, 1, P, D), -1.0)
    k[0, 0, 3] = -0.5                        # slot 3 has the largest logit of a positive row
    k[1, 0, 5] = -2.0                        # slot 21 that of a negative one
    v = torch.arange(3 * P).view(3, 1, P, 1).expand(3, 1, P, D) / 4.0
    for mag in (2.0 ** 110, 2.0 ** 118):
        ks = 2.0 ** 20 if e4 else 1.0
        cache = ta.PagedKVCache(*(x.contiguous().to(cdtype).cuda() for x in (k, v)),
                                *((torch.full((3, 1), ks, device="cuda"), torch.ones(3, 1, device="cuda")) if e4 else ()))
        q = torch.stack([torch.full((2, D), mag / ks), torch.full((2, D), -mag / ks)]).to(dtype).cuda()
        o, lse = ta.paged_attention(q, cache, _i32([[0, 1, 2], [0, 1, 2]]), _i32([n, n]), return_aux=True)
        torch.cuda.synchronize()
        assert ta.get_status() == 0
        for i, (slot, x) in enumerate(((3, -0.5), (21, 2.0))):
            assert bool((o[i].float() == v[slot // P, 0, slot % P].to(cdtype).to(dtype).float().cuda()).all()), (mag, i, o[i, 0, 0])
            want = x * mag * D ** 0.5
            assert bool(((lse[:, i].double() - want).abs() <= 2.0 ** -20 * abs(want)).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_value_scales_at_and_past_their_range(dtype):
    """2^-56 and 2^56 beside 1: every weight counts (32 equal logits, so each weight is 2^-5 and O the mean over pages);
    past them, zero, NaN and infinity: the page's slots are not seen, and the status says so."""
    import math

    import masked_attention_tri_gb300 as ta
    F8, D = torch.float8_e4m3fn, 64
    k = torch.zeros(3, 1, 16, D, device="cuda").to(F8)
    v = torch.ones(3, 1, 16, D, device="cuda").to(F8)
    ks = torch.ones(3, 1, device="cuda")
    q = torch.ones(1, 2, D, device="cuda").to(dtype)
    call = lambda vs, pages, n: ta.paged_attention(q, ta.PagedKVCache(k, v, ks, vs), _i32([pages]), _i32([n]), return_aux=True)  # noqa: E731
    for scale in (2.0 ** -56, 1.0, 2.0 ** 56):
        vs = torch.tensor([[1.0], [scale], [1.0]], device="cuda")
        o, lse = call(vs, [0, 1], 32)
        assert ta.get_status() == 0
        want = torch.tensor((1 + scale) / 2).to(dtype).float()       # (2^55 is an infinity in fp16)
        assert bool((o.float().cpu() == want).all()) or abs(float(o[0, 0, 0]) / float(want) - 1) <= 2.0 ** -11
        assert float((lse.double().cpu() - math.log(32)).abs().max()) <= 2.0 ** -19
    for bad in (2.0 ** -57, 2.0 ** 57, 1e-40, 0.0, -1.0, math.nan, math.inf):
        vs = torch.tensor([[1.0], [bad], [1.0]], device="cuda")
        o, lse = call(vs, [0, 1, 2], 48)
        assert ta.get_status() == abi.TA_ERR_DEVICE
        assert bool((o == 1).all()) and float((lse.double().cpu() - math.log(32)).abs().max()) <= 2.0 ** -19
        o, lse = call(vs, [1], 7)
        assert ta.get_status() == abi.TA_ERR_DEVICE and bool((o == 0).all()) and bool((lse == -math.inf).all())
        call(vs, [0, 2, 1], 32)                                      # a page that no row sees may have any
        assert ta.get_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_small_elements_of_a_query_over_8_bit_keys(dtype, D):
    """A query row whose elements span 2^-24 to 1, against keys whose codes grow as its elements shrink.  16-bit queries are
    scaled by a power of two, their largest magnitude into [1, 2), and held in fp16, whose least step there is 2^-24:
    an element is off by at most 2^-25 of the largest, a logit by scale 2^-25 max|q| sum|k|; fp32 queries by nothing.  The
    rest as in test_paged_attention.py: the products' sum D 2^-23 E, 2^-22 |x|, the logarithm's 2^-20."""
    import masked_attention_tri_gb300 as ta
    F8 = torch.float8_e4m3fn
    g = torch.Generator().manual_seed(D)
    i = torch.arange(D)
    size = torch.exp2(-24.0 * i / (D - 1))
    q = (size * torch.randn(1, 4, D, generator=g).sign() * (1 + torch.rand(1, 4, D, generator=g))).to(dtype)
    big = torch.exp2((i * 8 // D).float())                     # up to 2^7 where the query is smallest
    k = ((torch.rand(2, 1, 16, D, generator=g) + 0.5) * big * torch.randn(2, 1, 16, D, generator=g).sign()).to(F8)
    v = torch.ones(2, 1, 16, D).to(F8)
    cache = ta.PagedKVCache(k.cuda(), v.cuda(), torch.ones(2, 1, device="cuda"), torch.ones(2, 1, device="cuda"))
    _, lse = ta.paged_attention(q.cuda(), cache, _i32([[0, 1]]), _i32([32]), scale=1.0, return_aux=True)
    torch.cuda.synchronize()
    assert ta.get_status() == 0
    kk, qq = k.double().reshape(32, D), q.double()[0]
    x = qq @ kk.t()
    E = (qq.abs() @ kk.abs().t()).amax(-1)
    tol = D * 2.0 ** -23 * E + 2.0 ** -22 * x.abs().amax(-1) + 2.0 ** -20
    if dtype != torch.float32:
        tol = tol + 2.0 ** -25 * qq.abs().amax(-1) * kk.abs().sum(-1).amax()
    err = (lse[:, 0].double().cpu() - torch.logsumexp(x, -1)).abs()
    assert bool((err <= tol).all()), (err, tol)
