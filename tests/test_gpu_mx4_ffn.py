"""The experts' products with 4-bit operands on the GPU against the 64-bit
reference.  The elementwise bound comes with the reference (mx4_ref.ffn_bounded):
fp32 products and sums, SwiGLU values that such an error may carry over a
rounding boundary of the second quantisation, and two bf16 roundings."""
import numpy as np
import pytest
import torch

import dispatch_grouped_gemm_gb300 as hmm
from tests import mx4_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(T, H, I, E, K, seed=0, ids=None, wdtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16)
    if ids is None:
        ids = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)])
    w = torch.softmax(torch.randn((T, K), generator=g), 1).to(wdtype)
    W1 = (torch.randn((E, H, 2 * I), generator=g) * H ** -0.5).to(torch.bfloat16)
    W2 = (torch.randn((E, I, H), generator=g) * I ** -0.5).to(torch.bfloat16)
    return x, ids.to(torch.int32), w, W1, W2


def run(x, ids, w, W1, W2):
    up = hmm.mx4_quantize_experts(W1.to(DEV), gate_up=True)
    down = hmm.mx4_quantize_experts(W2.to(DEV))
    y = hmm.moe_ffn_mx4(x.to(DEV), ids.to(DEV), w.to(DEV), up, down)
    return y, up, down


def check(x, ids, w, W1, W2, tokens=None):
    y, up, down = run(x, ids, w, W1, W2)
    c = hmm.Context.for_device(y.device)
    assert hmm.hmm_status(c.handle) == (0, 0)
    y = y.double().cpu().numpy()
    V1 = up.dequantize(torch.float32).double().cpu().numpy()
    V2 = down.dequantize(torch.float32).double().cpu().numpy()
    t = np.arange(x.shape[0]) if tokens is None else tokens
    want, lim = ref.ffn_bounded(x.double().numpy()[t], ids.numpy()[t], w.double().numpy()[t],
                                V1, V2)
    bad = ~(np.abs(y[t] - want) <= lim)
    assert not bad.any(), (int(bad.sum()), bad.size, float((np.abs(y[t] - want) / lim).max()))
    # the bound itself has to say something
    assert np.median(lim / (np.abs(want) + 1e-9)) < 0.2


@pytest.mark.parametrize("T,H,I,E,K", [
    (1, 8, 8, 1, 1), (1, 32, 32, 4, 2), (3, 40, 24, 5, 2), (7, 64, 96, 3, 3), (16, 128, 64, 4, 1),
    (33, 264, 168, 6, 2), (65, 256, 128, 2, 2), (130, 520, 392, 3, 1), (64, 512, 256, 8, 2),
    (20, 1024, 288, 4, 4), (5, 776, 1032, 3, 2), (40, 288, 512, 40, 8), (2, 2048, 1408, 4, 2)])
def test_shapes(T, H, I, E, K):
    check(*make(T, H, I, E, K, seed=T + H))


@pytest.mark.parametrize("wdtype", [torch.float32, torch.bfloat16])
def test_hot_empty_and_ragged_experts(wdtype):
    """One expert with several token blocks, others with 0, 1, 127 .. 129 rows."""
    sizes = [300, 0, 1, 127, 128, 129, 0, 17, 33, 64]
    ids = torch.cat([torch.full((n,), e) for e, n in enumerate(sizes)])
    ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(1))].view(-1, 1)
    check(*make(len(ids), 256, 160, len(sizes), 1, ids=ids, wdtype=wdtype),
          tokens=np.arange(0, len(ids), 7))


def test_one_expert_many_times():
    """The same expert several times for one token (rows are separate slots)."""
    ids = torch.tensor([[2, 2, 2], [0, 2, 0], [1, 1, 1]])
    check(*make(3, 96, 64, 3, 3, ids=ids))
    check(*make(20, 320, 96, 3, 8, ids=torch.ones((20, 8), dtype=torch.long)))


@pytest.mark.parametrize("T,H,I,E,K", [(4096, 2048, 1408, 64, 6), (128, 1024, 512, 256, 8),
                                       (9000, 512, 256, 4, 2)])
def test_larger(T, H, I, E, K):
    check(*make(T, H, I, E, K, seed=3), tokens=np.random.default_rng(0).integers(0, T, 24))


@pytest.mark.parametrize("T,H,I,E,K", [(3637, 2064, 976, 24, 3), (2600, 6040, 696, 8, 2),
                                       (4000, 752, 1936, 32, 2), (1500, 4112, 520, 12, 4),
                                       (5000, 272, 136, 64, 4)])
def test_long_batch_like_short_ones(T, H, I, E, K):
    """A token's result does not depend on the other tokens, its place in a
    block or the tiles' width: a long batch gives bit for bit what batches of
    100 tokens give, call after call without a wait in between.  (Widths whose
    last tile is narrow mix tiles that share accumulator columns with tiles
    that do not.)"""
    x, ids, w, W1, W2 = (t.to(DEV) for t in make(T, H, I, E, K, seed=T))
    up, down = hmm.mx4_quantize_experts(W1, gate_up=True), hmm.mx4_quantize_experts(W2)
    want = torch.cat([hmm.moe_ffn_mx4(a.contiguous(), b.contiguous(), c.contiguous(), up, down)
                      for a, b, c in zip(x.split(100), ids.split(100), w.split(100))])
    torch.cuda.synchronize()
    got = [hmm.moe_ffn_mx4(x, ids, w, up, down) for _ in range(12)]
    for y in got:
        assert torch.equal(y, want)


@pytest.mark.parametrize("T,H,I,E,K,hot", [(2000, 2064, 2600, 2, 2, None),
                                           (5000, 2048, 2016, 5, 1, (0, 301, 4442, 257, 0)),
                                           (1900, 6032, 2928, 2, 2, None),
                                           (4096, 2048, 1416, 4, 2, (4096, 129, 1, 3966)),
                                           (3900, 2304, 2640, 2, 1, (128, 3772))])
def test_pairs_of_blocks(T, H, I, E, K, hot):
    """Many rows per expert run on pairs of blocks: experts without tokens, with
    one row, with an odd number of blocks, widths whose last tile is narrow.
    What the short batches give, bit for bit, and the formula's values."""
    ids = None
    if hot is not None:
        assert sum(hot) == T * K
        ids = torch.repeat_interleave(torch.arange(E), torch.tensor(hot))
        ids = ids.reshape(K, T).T.flip(0).contiguous()
    args = make(T, H, I, E, K, seed=T, ids=ids)
    check(*args, tokens=np.random.default_rng(1).integers(0, T, 12))
    x, ids, w, W1, W2 = (t.to(DEV) for t in args)
    up, down = hmm.mx4_quantize_experts(W1, gate_up=True), hmm.mx4_quantize_experts(W2)
    want = torch.cat([hmm.moe_ffn_mx4(a.contiguous(), b.contiguous(), c.contiguous(), up, down)
                      for a, b, c in zip(x.split(100), ids.split(100), w.split(100))])
    torch.cuda.synchronize()
    got = [hmm.moe_ffn_mx4(x, ids, w, up, down) for _ in range(12)]
    for y in got:
        assert torch.equal(y, want)


def test_repeatable_and_other_stream():
    args = make(500, 512, 384, 16, 4, seed=5)
    y, up, down = run(*args)
    x, ids, w = (t.to(DEV) for t in args[:3])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        z = hmm.moe_ffn_mx4(x, ids, w, up, down)
    s.synchronize()
    assert torch.equal(y, z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z = hmm.moe_ffn_mx4(x, ids, w, up, down)
    x.copy_(x.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(z, hmm.moe_ffn_mx4(x, ids, w, up, down)) and not torch.equal(z, y)


def test_pairs_in_a_graph_on_another_stream():
    x, ids, w, W1, W2 = (t.to(DEV) for t in make(2000, 2048, 2592, 2, 2, seed=4))
    up, down = hmm.mx4_quantize_experts(W1, gate_up=True), hmm.mx4_quantize_experts(W2)
    want = hmm.moe_ffn_mx4(x, ids, w, up, down)
    flipped = hmm.moe_ffn_mx4(x.flip(0), ids.flip(0), w.flip(0), up, down)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y = hmm.moe_ffn_mx4(x, ids, w, up, down)
    s.synchronize()
    assert torch.equal(y, want) and torch.equal(flipped, want.flip(0))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = hmm.moe_ffn_mx4(x, ids, w, up, down)
    for a in (x, ids, w):
        a.copy_(a.flip(0))
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, flipped)


def test_stale_workspace_does_not_matter():
    """Padding rows, unused scale bytes and stale tiles hold NaN patterns."""
    x, ids, w, W1, W2 = make(70, 288, 96, 6, 2, seed=8)
    y, up, down = run(x, ids, w, W1, W2)
    shape = hmm.make_shape(70, 288, 96, 6, 2, hmm.HMM_DTYPE_F32)
    ws = torch.full((hmm.hmm_mx4_workspace_size(shape),), 255, dtype=torch.uint8, device=DEV)
    z = torch.empty_like(y)
    c = hmm.Context.for_device(y.device)
    hmm.hmm_forward_mx4(c.handle, shape, x.to(DEV), ids.to(DEV), w.to(DEV), up.codes, up.scales,
                        down.codes, down.scales, z, ws)
    assert torch.equal(y, z)


def test_non_finite_tokens_stay_with_their_token():
    x, ids, w, W1, W2 = make(40, 256, 128, 4, 2, seed=9)
    y, up, down = run(x, ids, w, W1, W2)
    x[3, 17], x[20, 250] = float("nan"), float("inf")
    z = hmm.moe_ffn_mx4(x.to(DEV), ids.to(DEV), w.to(DEV), up, down)
    bad = torch.zeros(40, dtype=torch.bool, device=DEV)
    bad[3] = bad[20] = True
    assert torch.isnan(z[bad]).all() and torch.equal(z[~bad], y[~bad])


def test_ids_out_of_range_set_the_status():
    x, ids, w, W1, W2 = make(10, 64, 64, 4, 2)
    ids[4, 1] = 4
    run(x, ids, w, W1, W2)
    c = hmm.Context.for_device(torch.device(DEV, 0))
    assert hmm.hmm_status(c.handle) == (hmm.HMM_ERR_EXPERT_ID, hmm.HMM_STATUS_EXPERT_ID)


def test_a_wait_that_runs_out_is_reported():
    args = make(40, 256, 128, 4, 2, seed=9)
    want, up, down = run(*args)
    c = hmm.Context(torch.device(DEV, 0))
    shape = hmm.make_shape(40, 256, 128, 4, 2, hmm.HMM_DTYPE_F32)
    ws = torch.empty(hmm.hmm_mx4_workspace_size(shape), dtype=torch.uint8, device=DEV)
    y = torch.empty_like(want)
    x, ids, w = (t.to(DEV) for t in args[:3])
    call = (c.handle, shape, x, ids, w, up.codes, up.scales, down.codes, down.scales, y, ws)
    c.set_option(hmm.HMM_OPT_WAIT_BUDGET_NS, 20_000_000)
    c.set_option(hmm.HMM_OPT_INJECT_SKIP_READY, 1)
    hmm.hmm_forward_mx4(*call)
    assert hmm.hmm_status(c.handle) == (hmm.HMM_ERR_TIMEOUT, hmm.HMM_STATUS_TIMEOUT)
    hmm.hmm_forward_mx4(*call)
    assert hmm.hmm_status(c.handle) == (0, 0) and torch.equal(y, want)


@pytest.mark.parametrize("T,hot", [(2000, (2000, 2000)), (2000, (1999, 2001)),
                                   (2000, (129, 3871))])
def test_a_wait_that_runs_out_in_pairs_is_reported(T, hot):
    ids = torch.repeat_interleave(torch.arange(2), torch.tensor(hot)).reshape(2, T).T.contiguous()
    args = make(T, 2048, 2592, 2, 2, seed=9, ids=ids)
    want, up, down = run(*args)
    c = hmm.Context(torch.device(DEV, 0))
    shape = hmm.make_shape(T, 2048, 2592, 2, 2, hmm.HMM_DTYPE_F32)
    ws = torch.empty(hmm.hmm_mx4_workspace_size(shape), dtype=torch.uint8, device=DEV)
    y = torch.empty_like(want)
    x, ids, w = (t.to(DEV) for t in args[:3])
    call = (c.handle, shape, x, ids, w, up.codes, up.scales, down.codes, down.scales, y, ws)
    c.set_option(hmm.HMM_OPT_WAIT_BUDGET_NS, 20_000_000)
    c.set_option(hmm.HMM_OPT_INJECT_SKIP_READY, 1)
    hmm.hmm_forward_mx4(*call)
    assert hmm.hmm_status(c.handle) == (hmm.HMM_ERR_TIMEOUT, hmm.HMM_STATUS_TIMEOUT)
    hmm.hmm_forward_mx4(*call)
    assert hmm.hmm_status(c.handle) == (0, 0) and torch.equal(y, want)


def test_empty():
    x, ids, w, W1, W2 = make(4, 64, 64, 4, 2)
    y, up, down = run(x, ids, w, W1, W2)
    z = hmm.moe_ffn_mx4(x[:0].to(DEV), ids[:0].to(DEV), w[:0].to(DEV), up, down)
    assert z.shape == (0, 64)


def test_refusals():
    x, ids, w, W1, W2 = (t.to(DEV) for t in make(4, 64, 64, 4, 2))
    up, down = hmm.mx4_quantize_experts(W1, gate_up=True), hmm.mx4_quantize_experts(W2)
    ok = (x, ids, w, up, down)
    hmm.moe_ffn_mx4(*ok)
    for i, bad, err in [(0, x.float(), TypeError), (0, x[:3], ValueError), (0, x.cpu(), ValueError),
                        (0, x[:, ::2], ValueError), (1, ids.long(), TypeError),
                        (1, ids[:, :1], ValueError), (2, w.half(), TypeError),
                        (3, down, ValueError), (4, up, ValueError),
                        (3, hmm.mx4_quantize_experts(W1[:3], gate_up=True), ValueError),
                        (0, x.clone().requires_grad_(), RuntimeError),
                        (2, w.clone().requires_grad_(), RuntimeError)]:
        with pytest.raises(err):
            hmm.moe_ffn_mx4(*ok[:i], bad, *ok[i + 1:])
    shape = hmm.make_shape(4, 64, 64, 4, 2, hmm.HMM_DTYPE_F32)
    n = hmm.hmm_mx4_workspace_size(shape)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    y = torch.empty_like(x)
    c = hmm.Context.for_device(x.device)
    call = [c.handle, shape, x, ids, w, up.codes, up.scales, down.codes, down.scales, y, ws]
    for i, bad, code in [(1, hmm.make_shape(4, 64, 64, 4, 2, 1, shared=1), -1), (2, None, -1),
                         (5, None, -1), (10, ws[:n - 256], -5), (9, y.data_ptr() + 2, -4),
                         (1, hmm.make_shape(4, 60, 64, 4, 2, 1), -4)]:
        with pytest.raises(hmm.HmmError) as e:
            hmm.hmm_forward_mx4(*call[:i], bad, *call[i + 1:])
        assert e.value.code == code
    with pytest.raises(hmm.HmmError):
        hmm.hmm_mx4_workspace_size(hmm.make_shape(4, 64, 64, 4, 2, 1, shared=1))
