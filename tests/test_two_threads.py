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
