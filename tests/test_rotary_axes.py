"""Rotary positions with several axes: refusals and the axes of pairs on the CPU, values and gradients on the GPU.

The reference turns each pair in fp64 by its own axis' position; tolerances as in test_rotary.py (an axis changes only
which position a pair is multiplied with).
"""
import pytest
import torch

from masked_attention_tri_gb300 import abi, build
from test_rotary import A, _check, _inputs

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _turn64(x, positions, rotary, back=False):
    th = torch.tensor(rotary.theta, dtype=torch.float64)
    ang = positions.double().cpu()[rotary.pair_axes.long().cpu()].t() * th
    c, s = (ang.cos() * rotary.attention_factor)[:, None], (ang.sin() * rotary.attention_factor)[:, None]
    s = -s if back else s
    y, n = x.double().cpu().clone(), rotary.dim // 2
    i0, i1 = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if rotary.interleaved else (slice(0, n), slice(n, 2 * n))
    a, b = y[..., i0].clone(), y[..., i1].clone()
    mag = torch.zeros_like(y)
    mag[..., i0] = mag[..., i1] = a.abs() + b.abs()
    y[..., i0], y[..., i1] = a * c - b * s, a * s + b * c
    return y, mag * rotary.attention_factor


# ---------------------------------------------------------------------------- CPU

def test_axes_of_pairs():
    import masked_attention_tri_gb300 as ta
    r = ta.Rotary(16, sections=(2, 3, 3))
    assert r.pair_axes.tolist() == [0, 0, 1, 1, 1, 2, 2, 2] and r.theta == ta.Rotary(16).theta
    assert r.positions_shape(5) == (3, 5) and ta.Rotary(16).positions_shape(5) == (5,)
    r = ta.Rotary(16, sections=(4, 1, 3), section_layout="interleaved", section_frequencies="own", base=100.0)
    assert r.pair_axes.tolist() == [0, 1, 2, 0, 2, 0, 2, 0]
    want = [0 / 4, 0, 0 / 3, 1 / 4, 1 / 3, 2 / 4, 2 / 3, 3 / 4]
    assert r.theta == [100.0 ** -w for w in want]


@pytest.mark.parametrize("kw", [dict(sections=(4, 3)), dict(sections=(8, 0)), dict(sections=()), dict(sections=(9, -1)),
                                dict(sections=(4, 4), section_layout="other"), dict(section_frequencies="own"),
                                dict(sections=(4, 4), section_frequencies="other"),
                                dict(sections=(4, 4), section_frequencies="own", scaling="linear", factor=2.0)])
def test_sections_refused(kw):
    import masked_attention_tri_gb300 as ta
    with pytest.raises(ValueError):
        ta.Rotary(16, **kw)


def _call(**kw):
    args = dict(q=A, k=A, dtype=abi.TA_BF16, positions=A, num_axes=3, pair_axes=A, turns=A, rotary_dim=64, interleaved=0,
                mscale=1.0, inverse=0, total=4, Hq=4, Hk=2, D=64, q_row_stride=0, k_row_stride=0, q_out_row_stride=0,
                k_out_row_stride=0, q_out=A + 0x10000, k_out=A + 0x20000, stream=0)
    args.update(kw)
    return abi.tri_attn_rotary_axes(**args)


@pytest.mark.parametrize("kw,exc", [
    (dict(num_axes=0), ValueError), (dict(pair_axes=None), ValueError), (dict(pair_axes=A + 2), ValueError),
    (dict(q=0), ValueError), (dict(positions=0), ValueError), (dict(rotary_dim=63), ValueError),
    (dict(D=264, rotary_dim=8), NotImplementedError)])
def test_refused(kw, exc):
    with pytest.raises(exc):
        _call(**kw)


# ---------------------------------------------------------------------------- GPU

CASES = [
    # tokens, Hq, Hk, D, dim, sections, layout, frequencies, interleaved, dtype, scaling
    (1, 1, 1, 8, 8, (2, 1, 1), "blocks", "shared", False, BF, None),
    (77, 32, 8, 128, 128, (16, 24, 24), "blocks", "shared", False, BF, None),
    (130, 5, 1, 96, 64, (8, 12, 12), "interleaved", "shared", True, F16, "yarn"),
    (33, 4, 2, 256, 128, (20, 44), "interleaved", "own", False, BF, None),
    (19, 3, 1, 40, 18, (3, 3, 2, 1), "interleaved", "own", True, BF, None),   # one pair at a time
    (50, 2, 1, 64, 64, (32,), "blocks", "shared", False, F32, "linear"),      # one axis
    (3001, 6, 2, 64, 64, (10, 11, 11), "blocks", "own", False, F32, None),
]


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,Hq,Hk,D,dim,sections,layout,freq,inter,dtype,scaling", CASES)
def test_values_and_gradients(tokens, Hq, Hk, D, dim, sections, layout, freq, inter, dtype, scaling):
    import masked_attention_tri_gb300 as ta
    kw = {} if scaling is None else dict(scaling=scaling, factor=4.0, original_length=512)
    rot = ta.Rotary(dim, interleaved=inter, sections=sections, section_layout=layout, section_frequencies=freq,
                    device="cuda", **kw)
    q, k = (t.cuda() for t in _inputs(tokens, Hq, Hk, D, dtype)[:2])
    g = torch.Generator().manual_seed(7)
    pos = torch.randint(-2 ** 31, 2 ** 31, (len(sections), tokens), generator=g).to(torch.int32)
    pos[0, 0] = -2 ** 31
    for back, call in ((False, ta.rotary_embedding), (True, ta.rotary_embedding_backward)):
        got = call(q, k, pos.cuda(), rot)
        for x, y in zip((q, k), got):
            _check(y, *_turn64(x, pos, rot, back))
    qa = q.clone().requires_grad_()
    ta.rotary_embedding_autograd(qa, None, pos.cuda(), rot).backward(q)
    assert bool((qa.grad == ta.rotary_embedding_backward(q, None, pos.cuda(), rot)).all())


@pytest.mark.gpu
def test_equal_axes_are_one_axis():
    import masked_attention_tri_gb300 as ta
    q, k = (t.cuda() for t in _inputs(300, 4, 2, 128, BF)[:2])
    pos = torch.arange(300, dtype=torch.int32, device="cuda") * 37
    one, three = ta.Rotary(128, device="cuda"), ta.Rotary(128, sections=(20, 22, 22), device="cuda")
    for x, y in zip(ta.rotary_embedding(q, k, pos, one), ta.rotary_embedding(q, k, pos.expand(3, -1).contiguous(), three)):
        assert bool((x == y).all())


@pytest.mark.gpu
def test_python_refusals():
    import masked_attention_tri_gb300 as ta
    q = torch.zeros(4, 2, 64, dtype=BF, device="cuda")
    rot = ta.Rotary(64, sections=(10, 22), device="cuda")
    for pos in (torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda"),
                torch.zeros(2, 4, dtype=torch.int64, device="cuda")):
        with pytest.raises(ValueError):
            ta.rotary_embedding(q, None, pos, rot)
