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
