"""The router on the GPU against the 64-bit reference (tests/gate_ref.py).

Tolerances.  A score's error comes from the fp32 exponent l - m (relative
2^-24 |l - m|, with |l - m| <= 20 in these inputs: 1.2e-6), expf (2 ulp), the
sum of E terms and the division (about 10 roundings): below 4e-6 in all, so
5e-6 relative.  A gradient is a few products of such scores: 2e-5 of the sum
of its terms' magnitudes.  bf16 outputs add half an ulp, 2^-9 relative.
Selection is compared exactly where keys are exact (softmax by the logit), and
through its keys (within 1e-6) where they are rounded sums."""
import math

import numpy as np
import pytest
import torch

import dispatch_grouped_gemm_gb300 as hmm
from tests import gate_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def logits_of(T, E, dtype, seed=0, masked=False):
    g = torch.Generator().manual_seed(seed)
    l = (1.5 * torch.randn((T, E), generator=g)).clamp(-8, 8)
    if masked:
        l[torch.rand((T, E), generator=g) < 0.2] = -math.inf
        l[T // 2] = -math.inf
        l[0, :] = -math.inf
        l[0, E - 1] = 1.0
    return l.to(dtype)


def check_selection(ids, key, K, is_open, exact):
    T, E = key.shape
    assert ids.dtype == torch.int32
    ids = ids.cpu().numpy().astype(np.int64)
    if exact:
        assert np.array_equal(ids, ref.select(key, K, is_open))
        return ids
    assert ((ids >= 0) & (ids < E)).all()
    tol = 1e-6
    for t in range(T):
        assert len(set(ids[t])) == K
        chosen = key[t, ids[t]]
        assert is_open[t, ids[t]].all()
        assert all(a >= b - tol for a, b in zip(chosen, chosen[1:]))
        rest = is_open[t].copy()
        rest[ids[t]] = False
        assert not (key[t, rest] > chosen.min() + tol).any()
    return ids


def close(got, want, rel, mag=None, dtype=torch.float32):
    got = got.double().cpu().numpy()
    lim = rel * np.abs(want if mag is None else mag) + 1e-30
    if dtype == torch.bfloat16:
        lim = lim + 2.0 ** -8 * np.abs(want)
    bad = ~(np.abs(got - want) <= lim)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4])


def run(l, K, dtype=torch.float32, bias=None, ds=None, dw=None, **kw):
    x = l.to(DEV).requires_grad_()
    b = None if bias is None else bias.to(DEV)
    out = hmm.moe_gate(x, K, bias=b, weights_dtype=dtype, return_scores=ds is not None, **kw)
    loss_of = [out[1]] + ([out[2]] if ds is not None else [])
    grads = [dw.to(DEV).to(dtype)] + ([ds.to(DEV)] if ds is not None else [])
    (dl,) = torch.autograd.grad(loss_of, x, grads)
    return out, dl


def compare(T, E, K, score, dtype, groups=1, topk_groups=1, group_top=1, renorm=False, scale=1.0,
            biased=False, scored=False, masked=False, wdtype=torch.float32, seed=0):
    l = logits_of(T, E, dtype, seed, masked)
    g = torch.Generator().manual_seed(seed + 1)
    bias = torch.randint(-50, 51, (E,), generator=g) * 1e-3 if biased else None
    dw = torch.randn((T, K), generator=g).to(wdtype).float()
    ds = 0.1 * torch.randn((T, E), generator=g) if scored else None
    out, dl = run(l, K, wdtype, bias, ds, dw, score=score, groups=groups,
                  topk_groups=topk_groups, group_top=group_top, renormalize=renorm, scale=scale)
    l64 = l.double().numpy()
    key = ref.keys(l64, score, None if bias is None else bias.numpy(), group_top)
    is_open = ref.open_experts(key, groups, topk_groups, group_top)
    by_logit = score == "softmax" and bias is None and group_top == 1
    ids = check_selection(out[0], key, K, is_open, by_logit)
    p = ref.scores(l64, score)
    close(out[1].detach(), ref.weights(p, ids, renorm, scale), 5e-6, dtype=wdtype)
    if scored:
        close(out[2].detach(), p, 5e-6)
    assert dl.dtype == dtype and dl.shape == l.shape
    want, mag = ref.d_logits(l64, ids, dw.numpy(), None if ds is None else ds.numpy(), score,
                             renorm, scale)
    close(dl, want, 2e-5, mag, dtype)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 8, 2), (3, 31, 5), (33, 32, 32), (17, 33, 8),
                                   (65, 64, 6), (129, 100, 7), (31, 160, 6), (63, 256, 8),
                                   (9, 384, 8), (5, 511, 9), (7, 1000, 32), (6, 1024, 1)])
def test_shapes(score, dtype, T, E, K):
    compare(T, E, K, score, dtype, renorm=K > 1 and T % 2 == 1, scale=2.5, biased=T % 3 == 0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,topk_groups,group_top", [
    (256, 8, 4, 2), (160, 8, 3, 1), (96, 32, 5, 3), (64, 2, 1, 2), (33, 3, 2, 1), (27, 9, 9, 3),
    (1024, 16, 2, 2), (40, 1, 1, 7), (480, 4, 3, 2), (24, 8, 2, 1)])
def test_groups(score, E, groups, topk_groups, group_top):
    K = min(6, E // groups * topk_groups)
    for biased in (False, True):
        compare(70, E, K, score, torch.float32, groups, topk_groups, group_top, renorm=True,
                biased=biased, seed=E)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("groups", [1, 4])
def test_closed_experts(score, renorm, groups):
    compare(40, 64, 6, score, torch.float32, groups, 2 if groups > 1 else 1, renorm=renorm,
            scored=True, masked=True)
    compare(40, 64, 6, score, torch.bfloat16, groups, 2 if groups > 1 else 1, renorm=renorm,
            masked=True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_and_bf16_weights(score):
    compare(50, 96, 4, score, torch.float32, scored=True, wdtype=torch.bfloat16, scale=1.5)
    compare(50, 96, 4, score, torch.bfloat16, scored=True, renorm=True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K,groups,topk_groups,group_top", [
    (64, 6, 1, 1, 1), (8, 8, 1, 1, 1), (128, 8, 1, 1, 1), (100, 7, 5, 3, 2), (160, 6, 8, 3, 1),
    (256, 8, 8, 4, 2), (224, 32, 4, 3, 2), (300, 5, 1, 1, 1), (512, 9, 32, 5, 2), (384, 8, 8, 4, 1),
    (1024, 16, 16, 2, 2), (30, 3, 1, 1, 1), (96, 6, 4, 2, 3), (300, 8, 4, 2, 2), (60, 5, 10, 4, 1),
    (120, 4, 1, 1, 3)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_tokens_like_few(score, E, K, groups, topk_groups, group_top, dtype):
    """A long batch gives row by row what short ones give: same ids, weights
    and scores up to the order of their sums (1e-6), closed experts, equal
    keys, infinities and NaN among them."""
    T = 4103
    l = logits_of(T, E, dtype, E)
    l[5], l[6], l[7], l[8, 3], l[9, 2], l[10, :E // 2] = -math.inf, 0.0, -0.0, math.nan, math.inf, 2.0
    l[torch.rand((T, E), generator=torch.Generator().manual_seed(3)) < 0.05] = -math.inf
    l = l.to(DEV)
    bias = (torch.randint(-20, 21, (E,), generator=torch.Generator().manual_seed(4)) * 1e-3).to(DEV)
    for b in (None, bias):
        for renorm in (False, True):
            kw = dict(score=score, bias=b, groups=groups, topk_groups=topk_groups,
                      group_top=group_top, renormalize=renorm, scale=1.5)
            a = hmm.moe_gate(l, K, return_scores=True, **kw)
            parts = [hmm.moe_gate(x, K, return_scores=True, **kw) for x in l.split(1024)]
            want = [torch.cat(p) for p in zip(*parts)]
            # sums in another order move p + bias or p + p by a rounding: only
            # exact keys have to select the same
            exact = score == "sigmoid" and group_top <= 2 or b is None and group_top == 1
            same = (a[0] == want[0]).all(1)
            assert same.all() if exact else same.float().mean() > 0.995
            for i in (1, 2):
                x, y = a[i][same], want[i][same]
                assert torch.equal(torch.isnan(x), torch.isnan(y))
                assert torch.allclose(x, y, rtol=2e-6, atol=1e-12, equal_nan=True)
            no_scores = hmm.moe_gate(l, K, **kw)
            assert torch.equal(no_scores[0], a[0])
            odd = torch.empty((T, E + 3), dtype=dtype, device=DEV)[:, 3:]
            odd.copy_(l)
            assert torch.equal(hmm.moe_gate(odd, K, **kw)[0][same], a[0][same])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K", [(64, 6), (8, 8), (128, 8), (100, 7), (160, 6), (256, 32), (300, 5),
                                 (512, 9), (1024, 16), (31, 3)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_tokens_gradient_like_few(score, E, K, dtype):
    """The gradient of a long batch against that of short ones, with and without
    gradients of the scores and of the weights: sums in another order, 2e-5 of
    the largest gradient of a row; bf16 outputs one rounding."""
    T = 4099
    g = torch.Generator().manual_seed(E)
    l = logits_of(T, E, dtype, E)
    l[5], l[7] = -math.inf, 0.0
    l[torch.rand((T, E), generator=g) < 0.05] = -math.inf
    l = l.to(DEV)
    dw, ds = torch.randn((T, K), generator=g).to(DEV), 0.1 * torch.randn((T, E), generator=g).to(DEV)

    def grad(x, dw, ds, renorm):
        x = x.detach().requires_grad_()
        _, w, p = hmm.moe_gate(x, K, score=score, renormalize=renorm, scale=1.5,
                               return_scores=True)
        outs = [o for o, d in ((w, dw), (p, ds)) if d is not None]
        return torch.autograd.grad(outs, x, [d for d in (dw, ds) if d is not None])[0]

    for renorm in (False, True):
        for a, b in ((dw, ds), (dw, None), (None, ds)):
            got = grad(l, a, b, renorm).float()
            # (short ones in fp32, so that only one side is rounded)
            want = torch.cat([grad(x, None if a is None else a[i:i + 1024],
                                   None if b is None else b[i:i + 1024], renorm)
                              for i, x in zip(range(0, T, 1024), l.float().split(1024))])
            lim = 2e-5 * want.abs().amax(1, keepdim=True) + 1e-12
            if dtype == torch.bfloat16:
                lim = lim + 2.0 ** -8 * want.abs()
            assert ((got - want).abs() <= lim).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K,groups,topk_groups,group_top", [
    (32, 4, 2, 1, 2), (20, 5, 1, 1, 1), (72, 6, 3, 2, 2), (96, 6, 6, 4, 1), (180, 8, 4, 2, 2),
    (192, 8, 2, 1, 2), (192, 7, 32, 9, 1), (356, 8, 4, 3, 2), (384, 6, 3, 2, 2), (400, 8, 5, 2, 2),
    (640, 8, 5, 3, 2), (768, 10, 16, 4, 2), (1020, 8, 4, 1, 2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_tokens_every_lane_width(score, E, K, groups, topk_groups, group_top, dtype):
    """8 to 40 experts per lane; groups of several lanes, lanes of several groups."""
    test_many_tokens_like_few(score, E, K, groups, topk_groups, group_top, dtype)
    test_many_tokens_gradient_like_few(score, E, K, dtype)


def test_equal_keys_go_to_the_lowest_index():
    l = torch.zeros((3, 70), device=DEV)
    l[1, 40:] = 1.0
    l[2, ::2] = -0.0
    for score in ("softmax", "sigmoid"):
        ids, w = hmm.moe_gate(l, 4, score=score)
        assert ids.tolist() == [[0, 1, 2, 3], [40, 41, 42, 43], [0, 1, 2, 3]]
        assert (w[0] == w[0, 0]).all()


def test_lowest_values_and_infinities():
    """A logit of the type's lowest value is an ordinary, tiny score; -inf
    comes after it; NaN shows up in the weights."""
    low = torch.finfo(torch.float32).min
    l = torch.tensor([[-math.inf, low, 0.0, -math.inf], [math.nan, 0.0, 1.0, 2.0]], device=DEV)
    ids, w = hmm.moe_gate(l, 3)
    assert ids[0].tolist() == [2, 1, 0] and w[0].tolist() == [1.0, 0.0, 0.0]
    assert ids[1].tolist() == [0, 3, 2] and torch.isnan(w[1]).all()
    ids, w = hmm.moe_gate(l, 3, score="sigmoid")
    assert ids[1].tolist() == [0, 3, 2] and torch.isnan(w[1, 0]) and not torch.isnan(w[1, 1:]).any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_row_strides(dtype):
    wide = logits_of(37, 131, dtype, 5).to(DEV)
    for view in (wide[:, 3:99], wide[::2, 1:65], wide[:1, 7:72].expand(5, 65),
                 wide[:, :96].t().contiguous().t().contiguous()):
        a, b = hmm.moe_gate(view, 5), hmm.moe_gate(view.contiguous(), 5)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    x = wide[:, 3:99].detach().requires_grad_()
    y = x.detach().contiguous().requires_grad_()
    for score in ("softmax", "sigmoid"):
        gx, = torch.autograd.grad(hmm.moe_gate(x, 5, score=score)[1].sum(), x)
        gy, = torch.autograd.grad(hmm.moe_gate(y, 5, score=score)[1].sum(), y)
        assert torch.equal(gx, gy)


def test_differences():
    """The GPU's gradient against central differences of the GPU's forward
    (fp32, step 1e-2: truncation ~ h^2 = 1e-4, rounding ~ 1e-6 / 1e-2 = 1e-4,
    of terms of order 1 to 3: 1e-3)."""
    l = logits_of(6, 24, torch.float32, 11).to(DEV)
    # keep the selection fixed under the step
    l = l.clamp(-2, 1)
    l[:, :4] += 6.0
    dw = torch.randn((6, 4), generator=torch.Generator().manual_seed(2)).to(DEV)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            x = l.clone().requires_grad_()
            ids, w = hmm.moe_gate(x, 4, score=score, renormalize=renorm)
            g, = torch.autograd.grad(w, x, dw)
            order = ids.sort(1)

            def loss(v):
                i, w = hmm.moe_gate(v, 4, score=score, renormalize=renorm)
                back = i.sort(1)
                assert torch.equal(back[0], order[0])
                d = torch.zeros_like(dw).scatter_(1, back[1], dw.gather(1, order[1]))
                return (w.double() * d.double()).sum(1)

            for e in range(24):
                hi, lo = l.clone(), l.clone()
                hi[:, e] += 1e-2
                lo[:, e] -= 1e-2
                diff = (loss(hi) - loss(lo)) / (hi[:, e].double() - lo[:, e].double())
                assert (diff - g[:, e].double()).abs().max() < 1e-3


def test_partial_gradients_and_empty():
    l = logits_of(9, 40, torch.float32).to(DEV).requires_grad_()
    ids, w, p = hmm.moe_gate(l, 3, return_scores=True)
    a, = torch.autograd.grad(p.sum(), l, retain_graph=True)
    assert a.abs().max() < 1e-5  # the scores sum to 1
    b, = torch.autograd.grad(w.sum(), l)
    assert b.abs().max() > 1e-3
    ids, w = hmm.moe_gate(l[:0], 3)
    assert ids.shape == (0, 3) and w.shape == (0, 3)


def test_streams_and_graph():
    l = logits_of(300, 256, torch.float32).to(DEV)
    want = hmm.moe_gate(l, 8, score="sigmoid")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = hmm.moe_gate(l, 8, score="sigmoid")
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = hmm.moe_gate(l, 8, score="sigmoid")
    l.copy_(l.flip(1))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], hmm.moe_gate(l, 8, score="sigmoid")[0])


def test_large_offsets():
    """Rows whose elements lie past 2^31."""
    E, ld = 64, 1 << 20
    l = torch.zeros(((1 << 31) + 64 * ld) // ld + 1, ld, dtype=torch.bfloat16, device=DEV)[:, :E]
    T = l.shape[0]
    l.copy_(logits_of(T, E, torch.bfloat16, 9))
    a, b = hmm.moe_gate(l, 6), hmm.moe_gate(l.contiguous(), 6)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_refusals():
    l = torch.zeros((4, 32), device=DEV)
    for kw, code in [(dict(k=33), -2), (dict(k=0), -2), (dict(k=2, groups=5), -2),
                     (dict(k=9, groups=8, topk_groups=2), -2), (dict(k=1, groups=0), -2),
                     (dict(k=1, groups=4, topk_groups=5), -2), (dict(k=1, group_top=33), -2),
                     (dict(k=1, scale=math.inf), -1), (dict(k=1, scale=math.nan), -1)]:
        with pytest.raises(hmm.HmmError) as e:
            hmm.moe_gate(l, **kw)
        assert e.value.code == code
    with pytest.raises(hmm.HmmError):
        hmm.moe_gate(torch.zeros((2, 1025), device=DEV), 1)
    for bad in (l[0], l.t(), l.cpu()):
        with pytest.raises(ValueError):
            hmm.moe_gate(bad, 1)
    for bad in (l.half(), l.double()):
        with pytest.raises(TypeError):
            hmm.moe_gate(bad, 1)
    with pytest.raises(ValueError):
        hmm.moe_gate(l, 1, score="tanh")
    with pytest.raises(ValueError):
        hmm.moe_gate(l, 1, bias=torch.zeros(31, device=DEV))
    with pytest.raises(TypeError):
        hmm.moe_gate(l, 1, bias=torch.zeros(32, device=DEV, dtype=torch.bfloat16))
    c = hmm.Context.for_device(l.device)
    g = hmm.make_gate(4, 32, 2, logits_dtype=7)
    i, w = torch.zeros((4, 2), dtype=torch.int32, device=DEV), torch.zeros((4, 2), device=DEV)
    for args, code in [((g, l, None, i, w), -3), ((hmm.make_gate(4, 32, 2), None, None, i, w), -1),
                       ((hmm.make_gate(4, 32, 2, ld_logits=31), l, None, i, w), -2),
                       ((hmm.make_gate(4, 32, 2, score=3), l, None, i, w), -1),
                       ((hmm.make_gate(4, 32, 2), l.data_ptr() + 2, None, i, w), -4)]:
        with pytest.raises(hmm.HmmError) as e:
            hmm.hmm_gate_forward(c.handle, *args)
        assert e.value.code == code
