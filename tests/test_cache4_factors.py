"""Factors of a 4-bit cache at the ends of their range, 2^-100 and 2^100, and beyond it.

Rows are n s f for whole numbers n up to 7 (7 among them) and an e4m3 number s: they are held exactly and come back so, where
1 / f or 1 / (f s) past fp32's range gave other codes.
"""
import math

import pytest
import torch

from masked_attention_tri_gb300 import abi, build

F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _cache(factors, kind):
    import masked_attention_tri_gb300 as ta
    f = torch.tensor(factors, dtype=torch.float32, device="cuda")
    one = torch.ones_like(f)
    c = ta.PagedKVCache4.empty(2, len(factors), 16, 64, *((f, one) if kind == "k" else (one, f)))
    for t in (c.k, c.v, c.k_scale.view(torch.uint8), c.v_scale.view(torch.uint8)):
        t.fill_(0x11)
    return c, f


def _rows(f, dtype):
    g = torch.Generator(device="cuda").manual_seed(3)
    n = torch.randint(-7, 8, (20, f.numel(), 4, 16), generator=g, device="cuda").float()
    n[..., 0] = 7
    s = torch.exp2(torch.randint(-9, 9, (20, f.numel(), 4, 1), generator=g, device="cuda").float())
    return (n * s * f[:, None, None]).flatten(2).to(dtype)


def _tables():
    return (torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"), torch.tensor([20], dtype=torch.int32, device="cuda"),
            torch.tensor([0, 20], dtype=torch.int32, device="cuda"))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["k", "v"])
def test_ends_of_the_range(dtype, kind):
    import masked_attention_tri_gb300 as ta
    c, f = _cache([2.0 ** -100, 1.0, 2.0 ** 100], kind)
    x, plain = _rows(f, dtype), _rows(torch.ones_like(f), dtype)
    k, v = (x, plain) if kind == "k" else (plain, x)
    table, held, cu = _tables()
    ta.kv_cache_append(c, k, v, table, held, cu, 20)
    a, b = ta.kv_cache_read(c, table, held, cu, 20, 20, dtype=dtype)
    assert torch.equal(a, k) and torch.equal(b, v) and ta.get_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [2.0 ** -101, 2.0 ** -130, 2.0 ** 101, 0.0, -1.0, math.inf, math.nan])
@pytest.mark.parametrize("kind", ["k", "v"])
def test_out_of_range(bad, kind):
    """Nothing of those heads is written, and the status says so; the other tensor is."""
    import masked_attention_tri_gb300 as ta
    c, _ = _cache([1.0, bad], kind)
    x = _rows(torch.ones(2, device="cuda"), torch.bfloat16)
    table, held, cu = _tables()
    ta.get_status()
    ta.kv_cache_append(c, x, x, table, held, cu, 20)
    assert ta.get_status() == abi.TA_ERR_DEVICE
    codes, scale, other = (c.k, c.k_scale, c.v) if kind == "k" else (c.v, c.v_scale, c.k)
    assert bool((codes == 0x11).all()) and bool((scale.view(torch.uint8) == 0x11).all()) and not bool((other == 0x11).all())
