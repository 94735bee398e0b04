"""Calls of two host threads at once, of sizes that share a kernel but not its shared memory."""
import math
import threading

import pytest
import torch

from masked_attention_tri_gb300 import build


def _both(calls, times):
    """Each call `times` times in a thread and stream of its own; its last result, and the first error of any."""
    out, errors, start = [None] * len(calls), [], threading.Barrier(len(calls))

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                for _ in range(times):
                    out[i] = calls[i]()
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        raise errors[0]
    return out


@pytest.mark.gpu
def test_paged_attention():
    build.build()
    import masked_attention_tri_gb300 as ta
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table, held, calls = i32([[0, 1]]), i32([20]), []
    for D in (132, 256):
        cache = ta.PagedKVCache(*(torch.randn(2, 1, 16, D, device="cuda") for _ in range(2)))
        q = torch.randn(1, 2, D, device="cuda")
        calls.append(lambda q=q, cache=cache: ta.paged_attention(q, cache, table, held))
    want = [c() for c in calls]
    torch.cuda.synchronize()
    got = _both(calls, 3000)
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and ta.get_status() == 0


@pytest.mark.gpu
def test_packed_backward():
    """Lists of q blocks of different lengths; dQ's sums come in any order (one rounding of the result apart)."""
    build.build()
    import masked_attention_tri_gb300 as ta
    calls = []
    for L in (130, 4000):
        q, k, v, g = (torch.randn(L, 1, 128, device="cuda").to(torch.bfloat16) for _ in range(4))
        cu = torch.tensor([0, L], dtype=torch.int32, device="cuda")
        kw = dict(mask_mod="sliding_window", window=60)
        o, lse, _ = ta.varlen_attention(q, k, v, cu, cu, L, L, return_aux=True, **kw)
        calls.append(lambda a=(q, k, v, cu, cu, L, L, o, lse, g), kw=kw: ta.varlen_attention_backward(*a, **kw)[:3])
    want = [c() for c in calls]
    torch.cuda.synchronize()
    got = _both(calls, 1000)
    assert ta.get_status() == 0
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert math.isfinite(float(y.float().abs().max()))
            assert bool(((x.float() - y.float()).abs() <= 2.0 ** -7 * x.float().abs() + 2.0 ** -12).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,sizes", [(torch.float32, ((16, 40), (64, 128))), (torch.float32, ((16, 136), (64, 256))),
                                         (torch.bfloat16, ((16, 80), (16, 128))), (torch.bfloat16, ((16, 136), (16, 256))),
                                         (torch.float16, ((16, 16), (16, 64)))])
def test_triangle_attention(dtype, sizes):
    """(the C entry point: the less a call does besides, the likelier the two threads meet)"""
    build.build()
    import masked_attention_tri_gb300 as ta
    from masked_attention_tri_gb300 import abi
    from masked_attention_tri_gb300.api import _DT
    calls, outs, want = [], [], []
    for L, D in sizes:
        q, k, v = (torch.randn(1, 1, 1, L, D, device="cuda").to(dtype) for _ in range(3))
        bias, out = torch.randn(1, 1, 1, L, L, device="cuda").to(dtype), torch.zeros_like(q)
        want.append(ta.triangle_attention(q, k, v, bias, scale=0.1))
        a = [x.data_ptr() for x in (q, k, v)] + [_DT[dtype], bias.data_ptr(), _DT[dtype], 0, 0, 1, 1, 1, L, L, D, 0.1, out.data_ptr(), 0, 0]
        calls.append(lambda a=a, keep=(q, k, v, bias): abi.tri_attn_fwd(*a, torch.cuda.current_stream().cuda_stream))
        outs.append(out)
    torch.cuda.synchronize()
    _both(calls, 20000)
    assert all(torch.equal(a, b) for a, b in zip(want, outs)) and ta.get_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [((16, 16), (64, 128)), ((16, 136), (64, 256))])
def test_triangle_backward(sizes):
    build.build()
    import masked_attention_tri_gb300 as ta
    from masked_attention_tri_gb300 import abi
    calls, outs, want = [], [], []
    for L, D in sizes:
        q, k, v, g = (torch.randn(1, 1, 1, L, D, device="cuda") for _ in range(4))
        bias = torch.randn(1, 1, 1, L, L, device="cuda")
        o, lse, _ = ta.triangle_attention(q, k, v, bias, scale=0.1, return_aux=True)
        want.append(ta.triangle_attention_backward(q, k, v, bias, lse, g, scale=0.1))
        out, n = [torch.zeros_like(x) for x in (q, k, v, bias)], abi.tri_attn_bwd_workspace_size(1, 1, 1, L, L, D)
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        a = [x.data_ptr() for x in (q, k, v)] + [0, bias.data_ptr(), 0, 0, 0, 1, 1, 1, L, L, D, 0.1, lse.data_ptr(), 0, g.data_ptr()]
        a += [x.data_ptr() for x in out] + [ws.data_ptr(), n]
        calls.append(lambda a=a, keep=(q, k, v, g, bias, lse, ws): abi.tri_attn_bwd(*a, torch.cuda.current_stream().cuda_stream))
        outs.append(out)
    torch.cuda.synchronize()
    _both(calls, 10000)
    assert ta.get_status() == 0
    for a, b in zip(want, outs):
        for x, y in zip(a, b):  # dQ of two key tiles: two fp32 sums in either order
            assert bool(((x - y).abs() <= 2.0 ** -20 * x.abs().max()).all())


@pytest.mark.gpu
@pytest.mark.parametrize("D", [16, 128])
def test_packed_forward(D):
    build.build()
    import masked_attention_tri_gb300 as ta
    from masked_attention_tri_gb300 import abi
    calls, outs, want = [], [], []
    for lens in ([16], [20] * 1000):
        q, k, v = (torch.randn(sum(lens), 1, D, device="cuda").to(torch.bfloat16) for _ in range(3))
        cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
        want.append(ta.varlen_attention(q, k, v, cu, cu, max(lens), max(lens), scale=0.1, mask_mod="causal"))
        out, n, m = torch.zeros_like(q), sum(lens), max(lens)
        a = [x.data_ptr() for x in (q, k, v)] + [abi.TA_BF16, cu.data_ptr(), cu.data_ptr(), len(lens), n, n, m, m, 1, D, 0.1, 0, 0, 0, 0, 1, 0, 0,
                                                 128, 128, abi.TA_MASK_CAUSAL, out.data_ptr(), 0, 0]
        calls.append(lambda a=a, keep=(q, k, v, cu): abi.tri_attn_varlen_fwd(*a, torch.cuda.current_stream().cuda_stream))
        outs.append(out)
    torch.cuda.synchronize()
    _both(calls, 20000)
    assert all(torch.equal(a, b) for a, b in zip(want, outs)) and ta.get_status() == 0
