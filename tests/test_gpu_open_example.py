"""The example of experts built from the pieces: it runs, its layer's gradients are the
formula's, and its update moves each expert's matrix by the orthogonalised momentum."""
import math

import pytest
import torch

from examples import open_experts
from tests import open_ref as ref

pytestmark = pytest.mark.gpu


def test_runs():
    losses, layer = open_experts.main(steps=3)
    assert len(losses) == 3 and all(math.isfinite(v) for v in losses)
    assert all(bool(torch.isfinite(p).all()) for p in layer.parameters())


def test_gradients():
    """Against 64 bits: at most six roundings to bf16 on the way to a result, 2^-9 of its
    norm each, one doubled by the square and one for the results' own: 8 * 2^-9."""
    torch.manual_seed(1)
    T, H, I, E, K = 200, 64, 96, 6, 2
    layer = open_experts.OpenExperts(H, I, E, K)
    x = torch.randn((T, H), device="cuda").to(torch.bfloat16).requires_grad_()
    ids = torch.rand((T, E), device="cuda").argsort(1)[:, :K].int().contiguous()
    w = torch.rand((T, K), device="cuda").requires_grad_()
    dy = torch.randn((T, H), device="cuda").to(torch.bfloat16)
    got = torch.autograd.grad(layer.experts(x, ids, w), (x, w, layer.up, layer.down), dy)
    leaves = [t.detach().double().requires_grad_() for t in (x, w, layer.up, layer.down)]
    y = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for e in range(E):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        o = torch.relu(leaves[0][t] @ leaves[2][e]).square() @ leaves[3][e]
        y = y.index_add(0, t, o * leaves[1][t, k].unsqueeze(1))
    for g, want in zip(got, torch.autograd.grad(y, leaves, dy.double())):
        assert (g.double() - want).norm() <= 8 * 2.0 ** -9 * want.norm()


def test_update():
    """A first step from zero: p = -lr * sqrt(M / N) * X of (1 + momentum) g, whose scale
    falls away.  Of X's elements one in bf16 differs by the products' 35 * 2^-11 of the
    norm of its matrix at most; then the result rounds twice, 2^-8 of its size each."""
    torch.manual_seed(2)
    p = torch.nn.Parameter(torch.zeros((3, 48, 32), dtype=torch.bfloat16, device="cuda"))
    p.grad = torch.randn(p.shape, device="cuda").to(torch.bfloat16)
    open_experts.Muon([p], lr=0.5).step()
    want = -0.5 * 1.5 ** 0.5 * ref.orthogonalize(p.grad.double())
    err = (p.detach().double() - want).flatten(1).norm(dim=1)
    assert bool((err <= (35 * 2.0 ** -11 + 2 * 2.0 ** -8) * want.flatten(1).norm(dim=1)).all())
