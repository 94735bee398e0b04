"""Gradients that reach an autograd function as slices of another tensor: contiguous, but not on a 16-byte boundary.

torch.cat's gradients are such slices; each function's gradients have to be those of the same numbers in memory of their own.
"""
import pytest
import torch

from masked_attention_tri_gb300 import build
from masked_attention_tri_gb300.api import _dense

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("dtype", [BF, F16, F32])
def test_dense(dtype):
    x = torch.arange(65, dtype=F32).to(dtype)
    for t in (x[:64].view(8, 8), x[1:].view(8, 8), x[:64].view(8, 8).t(), x[:1].expand(8)):
        y = _dense(t)
        assert y.is_contiguous() and y.data_ptr() % 16 == 0 and torch.equal(y, t)
    assert _dense(x) is x


def _odd(outs, grads, leaves):
    """Gradients of the leaves where the outputs' gradients are slices behind one element."""
    one = torch.zeros(1, dtype=outs[0].dtype, device="cuda")
    flat = torch.cat([one] + [o.flatten() for o in outs])
    return torch.autograd.grad(flat, leaves, torch.cat([one] + [g.flatten() for g in grads]))


def _randn(*shape, dtype):
    return torch.randn(*shape, device="cuda").to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F16, F32])
def test_prompt(dtype):
    import masked_attention_tri_gb300 as ta
    torch.manual_seed(1)
    q, k, v, g = (_randn(70, h, 64, dtype=dtype) for h in (4, 2, 2, 4))
    cu = torch.tensor([0, 30, 70], dtype=torch.int32, device="cuda")
    leaves = [t.requires_grad_() for t in (q, k, v)]
    o = ta.prompt_attention_autograd(*leaves, cu, cu, 40, 40)
    want = torch.autograd.grad(o, leaves, g, retain_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(want, _odd([o], [g], leaves)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("with_k", [True, False])
def test_rotary(dtype, with_k):
    import masked_attention_tri_gb300 as ta
    torch.manual_seed(2)
    q, k, gq, gk = (_randn(33, h, 64, dtype=dtype) for h in (3, 1, 3, 1))
    pos = torch.arange(33, dtype=torch.int32, device="cuda")
    rot = ta.Rotary(64, device="cuda")
    leaves = [t.requires_grad_() for t in ((q, k) if with_k else (q,))]
    outs = ta.rotary_embedding_autograd(q, k if with_k else None, pos, rot)
    outs = list(outs) if with_k else [outs]
    grads = [gq, gk][:len(outs)]
    want = torch.autograd.grad(outs, leaves, grads, retain_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(want, _odd(outs, grads, leaves)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_triangle(dtype):
    import masked_attention_tri_gb300 as ta
    torch.manual_seed(3)
    q, k, v, g = (_randn(1, 2, 2, 64, 64, dtype=dtype) for _ in range(4))
    bias = _randn(1, 1, 2, 64, 64, dtype=F32)
    leaves = [t.requires_grad_() for t in (q, k, v)]
    o = ta.triangle_attention_autograd(*leaves, bias)
    want = torch.autograd.grad(o, leaves, g, retain_graph=True)
    # (64 keys: dQ is a sum of two addends at most, which has one result whatever their order)
    assert all(torch.equal(a, b) for a, b in zip(want, _odd([o], [g], leaves)))
