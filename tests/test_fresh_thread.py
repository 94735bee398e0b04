"""The library's call is the first thing that a host thread does with the GPU."""
import threading

import pytest
import torch

from masked_attention_tri_gb300 import abi, build

B16 = torch.bfloat16


def _in_thread(f):
    r = {}

    def work():
        try:
            f()
        except Exception as e:  # noqa: BLE001
            r["error"] = e
    t = threading.Thread(target=work)
    t.start()
    t.join()
    if "error" in r:
        raise r["error"]


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
def test_triangle(D):
    build.build()
    import masked_attention_tri_gb300 as ta
    q, k, v = (torch.randn(1, 2, 1, 40, D, device="cuda").to(B16) for _ in range(3))
    bias, out = torch.randn(1, 1, 1, 40, 40, device="cuda").to(B16), torch.zeros_like(q)
    want = ta.triangle_attention(q, k, v, bias)
    torch.cuda.synchronize()
    _in_thread(lambda: ta.triangle_attention(q, k, v, bias, out=out))
    torch.cuda.synchronize()
    assert torch.equal(out, want) and ta.get_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("mask", [dict(mask_mod="causal"), dict(mask_mod="sink_window", window=9, sinks=2)])
def test_packed(mask):
    build.build()
    import masked_attention_tri_gb300 as ta
    q, k, v = (torch.randn(300, 2, 64, device="cuda").to(B16) for _ in range(3))
    cu, out = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda"), torch.zeros_like(q)
    want = ta.varlen_attention(q, k, v, cu, cu, 200, 200, **mask)
    torch.cuda.synchronize()
    _in_thread(lambda: ta.varlen_attention(q, k, v, cu, cu, 200, 200, out=out, **mask))
    torch.cuda.synchronize()
    assert torch.equal(out, want) and ta.get_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,cdtype", [(B16, B16), (B16, torch.float8_e4m3fn), (torch.float32, torch.float32)])
def test_cache(dtype, cdtype):
    """Rows into the cache, rotated, and attention over them; the C entry points, with the workspace at hand."""
    build.build()
    import masked_attention_tri_gb300 as ta
    from masked_attention_tri_gb300.api import _DT
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    k, v, q = torch.randn(2, 1, 64, device="cuda").to(dtype), torch.randn(2, 1, 64, device="cuda").to(dtype), torch.randn(2, 4, 64, device="cuda").to(dtype)
    table, held, rot = i32([[0], [1]]), i32([1, 1]), ta.Rotary(64, device="cuda")
    caches = [ta.PagedKVCache.empty(2, 1, 16, 64, cdtype) for _ in range(2)]
    qr, out = torch.zeros_like(q), torch.zeros_like(q)
    n = abi.tri_attn_paged_workspace_size(_DT[dtype], 1, 4, 1, 64)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    want = ta.paged_attention(ta.kv_cache_append(caches[0], k, v, table, held, rotary=rot, q=q), caches[0], table, held)
    torch.cuda.synchronize()
    c, p = caches[1], lambda t: 0 if t is None else t.data_ptr()  # noqa: E731

    def append():
        ta.kv_cache_append(c, k, v, table, held, rotary=rot, q=q, out_q=qr)

    def attend():
        abi.tri_attn_paged_fwd(p(qr), _DT[dtype], 0, p(held), p(table), 2, 2, 1, 4, 1, 64, 0, 0.125, 0, 0, p(c.k), p(c.v), c._code,
                               p(c.k_scale), p(c.v_scale), 2, 16, 1, None, None, p(out), 0, p(ws), n, 0)
    _in_thread(append)
    _in_thread(attend)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and ta.get_status() == 0
