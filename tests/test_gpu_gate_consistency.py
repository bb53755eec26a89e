"""The router where scores are too small for fp32, where keys are rounded sums
and where arguments have no effect on the formula.  Tolerances as derived in
tests/test_gpu_gate.py."""
import math

import numpy as np
import pytest
import torch

import dispatch_grouped_gemm_gb300 as hmm
from tests import gate_ref as ref
from tests.test_gpu_gate import close, logits_of, run

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T", [5, 4100])
@pytest.mark.parametrize("E,K", [(64, 6), (33, 3), (300, 9)])
@pytest.mark.parametrize("scored", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_renormalised_weights_of_scores_below_fp32(T, E, K, scored, dtype):
    """A bias selects experts whose softmax scores underflow: their renormalised
    weights are the formula's, and the gradient is that of these weights.  (The
    selected logits lie within 20 of one another, as the tolerances assume.)"""
    g = torch.Generator().manual_seed(E)
    l = logits_of(T, E, dtype, E)
    few = torch.randperm(E, generator=g)[:K]
    l[:, few] = (-200.0 + l[:, few].float()).to(dtype)
    l[0, few[1:]] = -math.inf  # one selected expert that is open
    l[1] = -math.inf           # none
    l[2, few[0]] = 9.0         # one large score among those that underflow
    bias = torch.zeros(E)
    bias[few] = 4.0 + torch.arange(K).float()  # distinct keys
    dw = torch.randn((T, K), generator=g)
    ds = 0.1 * torch.randn((T, E), generator=g) if scored else None
    out, dl = run(l, K, torch.float32, bias, ds, dw, renormalize=True, scale=1.5)
    l64 = l.double().numpy()
    key = ref.keys(l64, "softmax", bias.numpy())
    ids = ref.select(key, K, np.ones((T, E), bool))
    assert np.array_equal(out[0].cpu().numpy(), ids)
    p = ref.scores(l64, "softmax")
    close(out[1].detach(), ref.weights(p, ids, True, 1.5), 5e-6)
    want, mag = ref.d_logits(l64, ids, dw.numpy(), None if ds is None else ds.numpy(), "softmax",
                             True, 1.5)
    assert np.abs(want[3:][:, few.numpy()]).max() > 0.01
    close(dl, want, 2e-5, mag, dtype)


@pytest.mark.parametrize("T", [3, 4100])
def test_group_top_has_no_effect_without_groups(T):
    """Logits whose softmax scores are equal in fp32: the selection goes by the
    logits, whatever group_top says of the one group."""
    l = (torch.arange(40, device=DEV) * 1e-9).expand(T, 40).contiguous()
    want = torch.arange(39, 33, -1, dtype=torch.int32, device=DEV).expand(T, 6)
    for top in (1, 2, 7):
        ids, w = hmm.moe_gate(l, 6, group_top=top)
        assert torch.equal(ids, want) and torch.allclose(w, torch.full_like(w, 1 / 40))


@pytest.mark.parametrize("E,K,groups,topk_groups,group_top", [
    (8, 3, 1, 1, 1), (64, 6, 1, 1, 1), (100, 7, 5, 3, 2), (128, 8, 1, 1, 1), (160, 6, 8, 3, 2),
    (164, 6, 1, 1, 1), (256, 8, 8, 4, 2), (260, 5, 1, 1, 1), (384, 8, 8, 4, 2), (512, 9, 32, 5, 2),
    (516, 9, 1, 1, 1), (768, 10, 16, 4, 2), (1024, 16, 1, 1, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_softmax_selection_does_not_depend_on_the_batch(E, K, groups, topk_groups, group_top, dtype):
    """Keys that are rounded sums, p + bias and sums of two p: the same experts
    and scores in a long batch, in short ones and for rows that are not aligned
    (all rows, ties and near ties among them)."""
    T = 4103
    l = logits_of(T, E, dtype, E)
    l[::3] = (l[::3] * 8).round() / 8  # many equal and nearly equal scores
    l[5], l[6] = -math.inf, 0.0
    l[torch.rand((T, E), generator=torch.Generator().manual_seed(3)) < 0.05] = -math.inf
    l = l.to(DEV)
    bias = (torch.randint(-20, 21, (E,), generator=torch.Generator().manual_seed(4)) * 1e-3).to(DEV)
    odd = torch.empty((T, E + 3), dtype=dtype, device=DEV)[:, 3:]
    odd.copy_(l)
    for b in (None, bias):
        kw = dict(bias=b, groups=groups, topk_groups=topk_groups, group_top=group_top,
                  return_scores=True)
        ids, w, p = hmm.moe_gate(l, K, **kw)
        short = [torch.cat(t) for t in zip(*(hmm.moe_gate(x, K, **kw) for x in l.split(1024)))]
        for other in (short, hmm.moe_gate(odd, K, **kw)):
            assert torch.equal(other[0], ids)
            if b is not None or group_top > 1:
                assert torch.equal(other[1], w) and torch.equal(other[2], p)


def test_second_derivatives_are_refused():
    """With create_graph the gradient is the same, and differentiating it raises
    (it would lose its dependence on the logits, silently beside other terms)."""
    l = logits_of(9, 40, torch.float32).to(DEV).requires_grad_()
    extra = torch.ones((), device=DEV, requires_grad=True)
    for through in (lambda out: out[1].sum(), lambda out: out[1].square().sum(),
                    lambda out: (out[2] * extra).square().sum()):
        for renorm in (False, True):
            kw = dict(renormalize=renorm, return_scores=True)
            want, = torch.autograd.grad(through(hmm.moe_gate(l, 3, **kw)), l)
            got, = torch.autograd.grad(through(hmm.moe_gate(l, 3, **kw)), l, create_graph=True)
            assert torch.equal(got, want)
            with pytest.raises(RuntimeError, match="moe_gate has no second derivative"):
                (got.square().sum() + extra).backward()


@pytest.mark.parametrize("T", [3, 4100])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_closed_logits_under_a_bias(T, score):
    """A logit of -inf has p = 0; its key is the bias, which may choose it, with
    weight 0 and no gradient; a bias of -inf closes an expert to every token."""
    l = torch.zeros((T, 8), device=DEV)
    l[:, 2:4] = -math.inf
    bias = torch.tensor([0.0, -2.0, 3.0, -1.0, -math.inf, -2.0, -2.0, -2.0], device=DEV)
    x = l.clone().requires_grad_()
    ids, w = hmm.moe_gate(x, 3, score=score, bias=bias)
    assert (ids == torch.tensor([2, 0, 3], device=DEV)).all()
    assert (w[:, 0] == 0).all() and (w[:, 1] > 0).all() and (w[:, 2] == 0).all()
    g, = torch.autograd.grad(w.sum(), x)
    assert (g[:, 2:4] == 0).all() and torch.isfinite(g).all() and (g[:, 0] > 0).all()
    ids, w = hmm.moe_gate(l, 8, score=score, bias=bias)
    assert (ids[:, 7] == 4).all()
    ids, w = hmm.moe_gate(l, 8, score=score)
    assert (ids == torch.tensor([0, 1, 4, 5, 6, 7, 2, 3], device=DEV)).all()
