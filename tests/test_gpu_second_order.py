"""moe_ffn under create_graph: the gradients are the same, and differentiating
them raises (they would lose their dependence on the arguments, silently beside
other terms)."""
import pytest
import torch

import dispatch_grouped_gemm_gb300 as hmm

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("shared", [False, True])
def test_second_derivatives_are_refused(shared):
    T, H, I, E, K = 20, 64, 32, 4, 2
    g = torch.Generator().manual_seed(1)

    def leaf(*shape, std=1.0, dtype=torch.bfloat16):
        return (std * torch.randn(shape, generator=g)).to(DEV, dtype).requires_grad_()

    x, w = leaf(T, H), leaf(T, K, dtype=torch.float32)
    W1, W2 = leaf(E, H, 2 * I, std=H ** -0.5), leaf(E, I, H, std=I ** -0.5)
    Ws = (leaf(H, 2 * I, std=H ** -0.5), leaf(I, H, std=I ** -0.5)) if shared else (None, None)
    ids = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]).int().to(DEV)
    inputs = [x, w, W1, W2] + [t for t in Ws if t is not None]

    def out():
        return hmm.moe_ffn(x, ids, w, W1, W2, shared_up_proj_weight=Ws[0],
                           shared_down_proj_weight=Ws[1]).float()

    for through in (lambda y: y.sum(), lambda y: y.square().sum()):
        want = torch.autograd.grad(through(out()), inputs)
        got = torch.autograd.grad(through(out()), inputs, create_graph=True)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
            with pytest.raises(RuntimeError, match="moe_ffn has no second derivative"):
                a.float().square().sum().backward(retain_graph=True)
        # one of several inputs
        got, = torch.autograd.grad(through(out()), W2, create_graph=True)
        assert torch.equal(got, want[3])
