"""Prompt attention over many key tiles, dS in two pieces, and calls of several threads and graphs at once.

Tolerances of values and gradients: test_prompt_attention.py's.
"""
import math

import pytest
import torch

from masked_attention_tri_gb300 import build
from test_fresh_thread import _in_thread
from test_prompt_attention import BF, F16, _cu, _i32, _inputs, _run, reference
from test_two_threads import _both

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


LONG = [
    # queries and keys of each sequence, Hq, Hk, D, dtype
    ([1100, 700, 520, 513, 511, 512, 640, 1], None, 8, 2, 96, BF),
    ([300, 900], [1700, 900], 8, 2, 96, F16),
    ([1300] * 8, None, 4, 4, 64, BF),                        # a CTA for each key tile walks all rows
    ([640, 639, 641, 768, 1025], None, 6, 2, 128, BF),       # 126 rows of a tile
    ([384], [2048], 5, 1, 72, BF),
    ([1000], [2500], 1, 1, 128, F16),
    ([2, 3, 900], [1500, 700, 901], 8, 1, 128, BF),
    ([700, 1500], [200, 1000], 4, 2, 64, BF),                # hundreds of rows without a key
    ([130] * 40, [700] * 40, 2, 1, 128, BF),
    ([1, 2, 127, 128, 129, 255, 256, 257, 383, 384, 385], [600, 640, 641, 768, 769, 895, 896, 897, 1023, 1024, 1025], 4, 1, 128,
     BF),
    ([48] * 11, [128 * i + 48 for i in range(11)], 16, 1, 64, F16),
]


@pytest.mark.parametrize("lq,lk,Hq,Hk,D,dtype", LONG)
def test_values_and_gradients(lq, lk, Hq, Hk, D, dtype):
    _run(lq, lk or lq, Hq, Hk, D, dtype)


@pytest.mark.parametrize("D,dtype", [(64, BF), (96, F16), (128, BF)])
def test_gradients_keep_their_own_rounding(D, dtype):
    """Of up to 512 keys dQ and dK are off by half a step of their own and by what fp32 sums and two 16-bit pieces of dS leave.

    The pieces: |dS| (eps / 2)^2 (in fp16 or its least step, 2^-25).  The rest as in test_prompt_attention.py with fp32's eps
    for P and the result: `reference` of the same numbers held in fp32.  A sum that lies that near a power of two may be rounded by
    the wider step beside it, to the power itself: off by twice that at most.
    """
    import masked_attention_tri_gb300 as ta
    lq = [512, 130, 301]
    q, k, v, g = _inputs(lq, lq, 4, 2, D, dtype)
    cu, s = _i32(_cu(lq)), float(torch.tensor(1 / math.sqrt(D), dtype=torch.float32))
    o, lse = ta.prompt_attention(q, k, v, cu, cu, 512, 512, return_aux=True)
    dq, dk, _ = ta.prompt_attention_backward(q, k, v, cu, cu, 512, 512, o, lse, g)
    R, T = reference(q.float(), k.float(), v.float(), lq, lq, s, g.float(), out=o.float())
    eps = torch.finfo(dtype).eps
    piece = {"dq": torch.zeros_like(R["dq"]), "dk": torch.zeros_like(R["dk"])}
    for a, b in zip(_cu(lq), _cu(lq)[1:]):
        hide = torch.ones(b - a, b - a, device="cuda").triu(1).bool()
        for h in range(4):
            Q, K, V, G = (x[a:b, i].double() for x, i in ((q, h), (k, h // 2), (v, h // 2), (g, h)))
            P = (s * (Q @ K.t())).masked_fill(hide, -math.inf).softmax(1)
            dS = P * (G @ V.t() - (G * o[a:b, h].double()).sum(1, keepdim=True))
            e = s * (dS.abs() * (eps / 2) ** 2 + (2.0 ** -25 if dtype == F16 else 0.0))
            piece["dq"][a:b, h] += e @ K.abs()
            piece["dk"][a:b, h // 2] += e.t() @ Q.abs()
    for name, x in (("dq", dq), ("dk", dk)):
        at = R[name].abs().clamp_min(torch.finfo(dtype).tiny)
        half = torch.exp2(torch.floor(torch.log2(at))) * eps / 2
        bad = (x.double() - R[name]).abs() > half + 2 * (T[name] + piece[name])
        assert not bool(bad.any()), (name, int(bad.sum()))
    assert ta.get_status() == 0


def _calls():
    """Calls of all operators and, for each kind, of sizes that differ (widths, tiles, workspaces)."""
    import masked_attention_tri_gb300 as ta
    sides = []
    for D, L, Hk, page in ((64, 70, 1, 16), (128, 900, 2, 64)):
        q, k, v, g = _inputs([L, 40], [L, 40], 4 * Hk, Hk, D, BF)
        cu = _i32([0, L, L + 40])
        pages = -(-L // page) + -(-40 // page)
        table = torch.zeros(2, -(-L // page), dtype=torch.int32, device="cuda")
        table[0] = torch.arange(table.shape[1])
        table[1, :-(-40 // page)] = torch.arange(table.shape[1], pages)
        held = _i32([L, 40])
        rotary = ta.Rotary(D, sections=(D // 4, D // 8, D // 8), device="cuda")
        positions = torch.randint(0, 99999, (3, L + 40), dtype=torch.int32, device="cuda")
        newest = torch.tensor([L - 1, L + 39], device="cuda")

        def work(q=q, k=k, v=v, g=g, cu=cu, pages=pages, table=table, held=held, rotary=rotary, positions=positions,
                 newest=newest, L=L, page=page):
            cache = ta.PagedKVCache4.empty(pages, k.shape[1], page, k.shape[2])
            qr = ta.kv_cache_append(cache, k, v, table, held, cu, L, rotary=rotary, positions=positions, q=q)
            kb, vb = ta.kv_cache_read(cache, table, held, cu, L, L + 40)
            o, lse = ta.prompt_attention(qr, kb, vb, cu, cu, L, L, return_aux=True)
            d = ta.prompt_attention_backward(qr, kb, vb, cu, cu, L, L, o, lse, g)
            back = ta.rotary_embedding_backward(d[0], d[1], positions, rotary)
            last = ta.paged_attention(qr.index_select(0, newest), cache, table, held)
            return (qr, kb, vb, o, lse, *d, *back, last)
        sides.append(work)
    return sides


def test_two_threads():
    import masked_attention_tri_gb300 as ta
    calls = _calls()
    want = [c() for c in calls]
    torch.cuda.synchronize()
    got = _both(calls, 150)
    for w, x in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, x))
    assert ta.get_status() == 0


def test_two_graphs_at_once():
    """Each graph keeps workspaces of its own: replayed in two streams at a time they do not meet."""
    import masked_attention_tri_gb300 as ta
    calls = _calls()
    want = [c() for c in calls]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for c, s in zip(calls, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs.append(c())
        graphs.append(graph)
    for _ in range(20):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for w, x in zip(want, outs):
        assert all(torch.equal(a, b) for a, b in zip(w, x))
    assert ta.get_status() == 0


def test_fresh_threads():
    calls = _calls()
    for c in calls:
        want, got = c(), []
        torch.cuda.synchronize()
        _in_thread(lambda c=c, got=got: got.extend(c()))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_any_upper_bound_of_the_lengths():
    """max_seqlen is an upper bound: one beyond the rows there are, or beyond int32, is as good as the longest length."""
    import masked_attention_tri_gb300 as ta
    lq = [70, 130]
    q, k, v, g = _inputs(lq, lq, 4, 2, 64, BF)
    cu, most = _i32(_cu(lq)), 2 ** 32 + 5
    o, lse = ta.prompt_attention(q, k, v, cu, cu, 130, 130, return_aux=True)
    o2, lse2 = ta.prompt_attention(q, k, v, cu, cu, most, most, return_aux=True)
    d = ta.prompt_attention_backward(q, k, v, cu, cu, 130, 130, o, lse, g)
    d2 = ta.prompt_attention_backward(q, k, v, cu, cu, most, most, o, lse, g)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and all(torch.equal(a, b) for a, b in zip(d, d2))
    cache = ta.PagedKVCache4.empty(4, 2, 64, 64)
    table, held = _i32([[0, 1, 0], [1, 2, 3]]), _i32([70, 130])
    ta.kv_cache_append(cache, k[70:], v[70:], table[1:], held[1:], _i32([0, 130]), 130)
    a = ta.kv_cache_read(cache, table[1:], held[1:], _i32([0, 130]), 130, 130)
    b = ta.kv_cache_read(cache, table[1:], held[1:], _i32([0, 130]), most, 130)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    # pages may be read by several sequences, and twice by one
    twice = ta.kv_cache_read(cache, _i32([[1, 1], [1, 2]]), _i32([128, 128]), _i32([0, 128, 256]), 128, 256)
    for x, y in zip(twice, a):
        assert torch.equal(x[:64], y[:64]) and torch.equal(x[64:128], y[:64]) and torch.equal(x[128:], y[:128])
    assert ta.get_status() == 0


def test_one_leaf_alone_and_through_rotation():
    """Gradients where one input asks for them, and along the chain rotation -> attention."""
    import masked_attention_tri_gb300 as ta
    lq = [200, 31]
    q, k, v, g = _inputs(lq, lq, 4, 2, 64, BF)
    cu = _i32(_cu(lq))
    rotary = ta.Rotary(64, sections=(16, 8, 8), device="cuda")
    positions = torch.randint(0, 5000, (3, 231), dtype=torch.int32, device="cuda")
    qr, kr = ta.rotary_embedding(q, k, positions, rotary)
    o, lse = ta.prompt_attention(qr, kr, v, cu, cu, 200, 200, return_aux=True)
    dq, dk, dv = ta.prompt_attention_backward(qr, kr, v, cu, cu, 200, 200, o, lse, g)
    dq, dk = ta.rotary_embedding_backward(dq, dk, positions, rotary)
    for ask in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 1)):
        leaves = [t.clone().requires_grad_(bool(a)) for t, a in zip((q, k, v), ask)]
        turned = ta.rotary_embedding_autograd(leaves[0], leaves[1], positions, rotary)
        ta.prompt_attention_autograd(*turned, leaves[2], cu, cu, 200, 200).backward(g)
        for leaf, a, want in zip(leaves, ask, (dq, dk, dv)):
            assert torch.equal(leaf.grad, want) if a else leaf.grad is None
