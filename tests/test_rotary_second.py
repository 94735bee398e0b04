"""Second derivatives through rotary positions."""
import pytest
import torch

from masked_attention_tri_gb300 import build


def _turn(x, pos, rot):
    """The turn in fp64 torch operations (interleaved pairs or halves), differentiable."""
    half, D = rot.dim // 2, x.shape[2]
    ang = pos.double().cpu()[:, None] * torch.tensor(rot.theta, dtype=torch.float64)
    c, s = (ang.cos() * rot.attention_factor)[:, None], (ang.sin() * rot.attention_factor)[:, None]
    t = x[..., :rot.dim]
    a, b = (t[..., 0::2], t[..., 1::2]) if rot.interleaved else (t[..., :half], t[..., half:])
    y, z = a * c - b * s, a * s + b * c
    t = torch.stack((y, z), -1).flatten(-2) if rot.interleaved else torch.cat((y, z), -1)
    return torch.cat((t, x[..., rot.dim:]), -1) if rot.dim < D else t


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("with_k", [False, True])
def test_second_derivatives(inter, with_k):
    """Of sum y^3 + sum y^2 w (w a leaf as well), against fp64 autograd: fp32 turns are off by 2^-22 of a pair (two
    products, their sum, and cos and sin), so a chain of four turns of values below 2^4 by less than 2^-14 of the
    largest second derivative."""
    build.build()
    import masked_attention_tri_gb300 as ta
    rot = ta.Rotary(16, interleaved=inter, scaling="yarn", factor=4.0, original_length=64, device="cuda")
    pos = torch.tensor([5, 0, -3, 1000], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(3)
    q, k, w = (torch.randn(4, h, 24, generator=g) for h in (2, 1, 2))

    def second(turn, q, k, w):
        q, k, w = (x.requires_grad_(True) for x in (q, k, w))
        y, z = turn(q, k)
        loss = (y ** 3).sum() + (y ** 2 * w).sum() + ((z ** 3).sum() if with_k else 0)
        leaves = (q, k, w) if with_k else (q, w)
        first = torch.autograd.grad(loss, leaves, create_graph=True)
        return torch.autograd.grad(sum((x ** 2).sum() for x in first), leaves)

    def ours(q, k):
        return ta.rotary_embedding_autograd(q, k, pos, rot) if with_k else (ta.rotary_embedding_autograd(q, None, pos, rot), None)

    got = second(ours, *(x.cuda() for x in (q, k, w)))
    want = second(lambda q, k: (_turn(q, pos, rot), _turn(k, pos, rot)), *(x.double() for x in (q, k, w)))
    assert ta.get_status() == 0
    for a, b in zip(got, want):
        assert float(b.abs().max()) > 1 and float((a.double().cpu() - b).abs().max()) <= 2.0 ** -14 * float(b.abs().max())
