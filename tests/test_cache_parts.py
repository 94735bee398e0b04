"""The tensors of a cache are public attributes: what a call uses is what stands there, and copies hold copies."""
import copy
import io
import pickle

import pytest
import torch

from masked_attention_tri_gb300 import build
from masked_attention_tri_gb300.cache import PagedKVCache, PagedKVCache4

U8, F8 = torch.uint8, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _parts4(pages=3, heads=2, page=16, D=32, device="cpu"):
    k, v = (torch.randint(0, 256, (pages, heads, page, D // 2), dtype=U8, device=device) for _ in range(2))
    ks, vs = ((torch.rand(pages, heads, page, D // 16, device=device) + 0.5).to(F8) for _ in range(2))
    return dict(k=k, v=v, k_scale=ks, v_scale=vs, k_factor=torch.full((heads,), 2.0, device=device),
                v_factor=torch.full((heads,), 0.5, device=device))


def _held(c):
    """The addresses that a call hands over."""
    return c._c.k, c._c.v, c._c.k_scale, c._c.v_scale, c._c.k_factor, c._c.v_factor, c._c.num_pages


def _own(c):
    return tuple(getattr(c, n).data_ptr() for n in ("k", "v", "k_scale", "v_scale", "k_factor", "v_factor")) + (c.num_pages,)


@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale", "k_factor", "v_factor"])
def test_another_tensor(name):
    c = PagedKVCache4(**_parts4())
    setattr(c, name, _parts4()[name])
    c._now()
    assert _held(c) == _own(c)
    getattr(c, name).data = _parts4()[name]  # the same tensor, other memory
    c._now()
    assert _held(c) == _own(c)


def test_a_cache_of_other_sizes():
    c = PagedKVCache4(**_parts4())
    for n, t in _parts4(pages=5, heads=4, page=32, D=64).items():
        setattr(c, n, t)
    c._now()
    assert _held(c) == _own(c) and (c.num_pages, c.heads, c.page_size, c.head_dim) == (5, 4, 32, 64)
    c.k_factor = None
    c._now()
    assert not c._c.k_factor


@pytest.mark.parametrize("name,other,exc", [
    ("k", None, TypeError), ("k", torch.zeros(3, 2, 16, 16), TypeError), ("k", torch.zeros(2, 2, 16, 16, dtype=U8), ValueError),
    ("v", torch.zeros(3, 2, 16, 32, dtype=U8), ValueError), ("v_scale", torch.zeros(3, 2, 16, 1).to(F8), ValueError),
    ("k_factor", torch.ones(3), ValueError)])
def test_another_tensor_that_does_not_fit(name, other, exc):
    c = PagedKVCache4(**_parts4())
    setattr(c, name, other)
    for _ in range(2):  # each call looks
        with pytest.raises(exc):
            c._now()


def test_expanded_tensors_are_refused():
    """One page that stands for all of them: its strides of 0 must not be taken for those of a contiguous cache."""
    one = _parts4(pages=1, heads=1)
    whole = {n: t.expand(3, 2, *t.shape[2:]) if t.dim() == 4 else None for n, t in one.items()}
    with pytest.raises(ValueError):
        PagedKVCache4(**whole)
    for n in ("k", "v", "k_scale", "v_scale"):
        for shape in ((3, 1), (1, 2)):  # pages, then heads
            parts = _parts4(pages=shape[0], heads=shape[1])
            t = parts[n][:1, :1].expand(*shape, *parts[n].shape[2:])
            with pytest.raises(ValueError):
                PagedKVCache4(**{**parts, "k_factor": None, "v_factor": None, n: t})
    whole = _parts4(pages=6)
    every_second = {n: t[::2] if t.dim() == 4 else t for n, t in whole.items()}
    assert list(PagedKVCache4(**every_second)._c.strides)[:2] == [2 * 2 * 16 * 16, 16 * 16]


def _pickled(c):
    f = io.BytesIO()
    pickle.dump(c, f)
    return pickle.loads(f.getvalue())


@pytest.mark.parametrize("how", [copy.deepcopy, copy.copy, _pickled])
def test_copies(how):
    parts = _parts4()
    c = PagedKVCache4(**parts)
    d = how(c)
    d._now()
    assert _held(d) == _own(d) and _held(c) == _own(c)
    for n, t in parts.items():
        x = getattr(d, n)
        assert torch.equal(x.view(U8) if t.dtype == F8 else x, t.view(U8) if t.dtype == F8 else t)
        assert (x.data_ptr() == t.data_ptr()) == (how is copy.copy)


def _parts(dtype, pages=3, heads=2, page=16, D=32, device="cpu"):
    if dtype == F8:
        k, v = (torch.randn(pages, heads, page, D, device=device).to(F8) for _ in range(2))
        return dict(k=k, v=v, k_scale=torch.ones(pages, heads, device=device), v_scale=torch.ones(pages, heads, device=device))
    return dict(zip("kv", (torch.randn(pages, heads, page, D, device=device).to(dtype) for _ in range(2))))


@pytest.mark.parametrize("dtype", [torch.bfloat16, F8, torch.float32])
def test_a_wider_cache_of_other_sizes(dtype):
    """Fewer pages, another page size, strided pages and another type: the next call counts them anew."""
    c = PagedKVCache(**_parts(F8))
    for n in ("k", "v", "k_scale", "v_scale"):
        setattr(c, n, _parts(dtype, 2, 4, 32, 64).get(n))
    c._now()
    assert (c.num_pages, c.heads, c.page_size, c.head_dim, c.dtype) == (2, 4, 32, 64, dtype) and c._strides == (None, None)
    both = torch.stack([_parts(dtype, 5, 4, 32, 64)["k"] for _ in range(2)], 1)  # the halves of one buffer
    c.k, c.v = both[:, 0], both[:, 1]
    if dtype == F8:
        c.k_scale, c.v_scale = torch.ones(5, 4), torch.ones(5, 4)
    c._now()
    assert c.num_pages == 5 and list(c._strides[0]) == [2 * 4 * 32 * 64, 32 * 64, 64]
    c.k = c.k[:4]
    for _ in range(2):
        with pytest.raises(ValueError):
            c._now()


@pytest.mark.parametrize("dtype", [torch.bfloat16, F8, torch.float32])
@pytest.mark.parametrize("how", [copy.deepcopy, copy.copy, _pickled])
def test_copies_of_a_wider_cache(dtype, how):
    both = torch.stack([_parts(dtype)["k"] for _ in range(2)], 1)
    c = PagedKVCache(**{**_parts(dtype), "k": both[:, 0], "v": both[:, 1]})
    d = how(c)
    d._now()
    assert torch.equal(d.k.float(), c.k.float()) and torch.equal(d.v.float(), c.v.float()) and d.num_pages == c.num_pages
    assert (d.k.data_ptr() == c.k.data_ptr()) == (how is copy.copy)
    assert all(tuple(a) == tuple(b) for a, b in zip(c._strides, d._strides))


@pytest.mark.gpu
def test_calls_use_what_stands_there():
    import masked_attention_tri_gb300 as ta
    torch.manual_seed(4)
    a, b = _parts4(device="cuda"), _parts4(pages=7, device="cuda")
    table = torch.tensor([[0, 2, 1]], dtype=torch.int32, device="cuda")
    held, cu = torch.tensor([40], dtype=torch.int32, device="cuda"), torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 4, 32, device="cuda").bfloat16()
    rows = torch.randn(1, 2, 32, device="cuda").bfloat16()
    want = ta.PagedKVCache4(**{n: t.clone() for n, t in b.items()})
    c = ta.PagedKVCache4(**a)
    ta.kv_cache_read(c, table, held, cu, 40, 40)
    before = {n: t.clone() for n, t in a.items()}
    for n, t in b.items():
        setattr(c, n, t)
    d = copy.deepcopy(c)
    for x in (want, c, d):
        ta.kv_cache_append(x, rows, rows, table, held)
    outs = [(*ta.kv_cache_read(x, table, held, cu, 40, 40), ta.paged_attention(q, x, table, held)) for x in (want, c, d)]
    for got in outs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(outs[0], got))
    for n, t in a.items():  # the old memory is left alone
        assert torch.equal(t.view(U8), before[n].view(U8))
    assert ta.get_status() == 0
