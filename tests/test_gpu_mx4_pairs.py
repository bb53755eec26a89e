"""The 4-bit expert products on CTA pairs, chosen by HMM_OPT_PAIR_ROWS whatever
the shape: bit for bit what single CTAs give, also at the shapes that the
automatic choice keeps on single CTAs (contractions of one K block, experts of
one row, one narrow tile of weight rows)."""
import numpy as np
import pytest
import torch

import dispatch_grouped_gemm_gb300 as hmm
from tests import mx4_ref as ref
from tests.test_gpu_mx4_ffn import make

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture
def context():
    c = hmm.Context(torch.device(DEV, 0))
    yield c
    c.close()


def call(c, mode, x, ids, w, up, down):
    c.set_option(hmm.HMM_OPT_PAIR_ROWS, mode)
    shape = hmm.make_shape(*x.shape, up.rows // 2, up.batch, ids.shape[1], hmm.HMM_DTYPE_F32)
    # (stale bytes are NaN patterns)
    ws = torch.full((hmm.hmm_mx4_workspace_size(shape),), 255, dtype=torch.uint8, device=DEV)
    y = torch.full_like(x, float("nan"))
    hmm.hmm_forward_mx4(c.handle, shape, x, ids, w, up.codes, up.scales, down.codes, down.scales,
                        y, ws)
    assert hmm.hmm_status(c.handle) == (0, 0)
    return y


@pytest.mark.parametrize("T,H,I,E,K,hot", [
    (1, 8, 8, 1, 1, None), (1, 32, 32, 4, 2, None), (3, 40, 24, 5, 2, None),
    (33, 264, 168, 6, 2, None), (65, 256, 128, 2, 2, None), (130, 520, 392, 3, 1, None),
    (20, 1024, 288, 4, 4, None), (40, 288, 512, 40, 8, None), (300, 2056, 32, 3, 2, None),
    (732, 256, 160, 10, 1, (300, 0, 1, 127, 128, 129, 0, 17, 0, 30)),
    (1024, 2304, 544, 4, 1, (257, 256, 255, 256)), (2000, 2064, 2600, 2, 2, None)])
def test_pairs_like_single_ctas(context, T, H, I, E, K, hot):
    ids = None
    if hot is not None:
        ids = torch.repeat_interleave(torch.arange(E), torch.tensor(hot)).view(T, K)
    host = make(T, H, I, E, K, seed=T + H, ids=ids)
    x, ids, w, W1, W2 = (t.to(DEV) for t in host)
    up, down = hmm.mx4_quantize_experts(W1, gate_up=True), hmm.mx4_quantize_experts(W2)
    want = call(context, 0, x, ids, w, up, down)
    for mode in (1, 1, 2, 3):
        assert torch.equal(call(context, mode, x, ids, w, up, down), want)
    t = np.arange(0, T, max(1, T // 8))
    y, lim = ref.ffn_bounded(host[0].double().numpy()[t], host[1].numpy()[t],
                             host[2].double().numpy()[t],
                             up.dequantize(torch.float32).double().cpu().numpy(),
                             down.dequantize(torch.float32).double().cpu().numpy())
    assert (np.abs(want.double().cpu().numpy()[t] - y) <= lim).all()


@pytest.mark.parametrize("T,H,I,E,K", [(1, 64, 32, 2, 1), (129, 264, 168, 2, 1),
                                       (700, 1024, 512, 4, 2)])
def test_a_wait_that_runs_out_is_reported(context, T, H, I, E, K):
    x, ids, w, W1, W2 = (t.to(DEV) for t in make(T, H, I, E, K, seed=9))
    up, down = hmm.mx4_quantize_experts(W1, gate_up=True), hmm.mx4_quantize_experts(W2)
    want = call(context, 0, x, ids, w, up, down)
    context.set_option(hmm.HMM_OPT_PAIR_ROWS, 1)
    context.set_option(hmm.HMM_OPT_WAIT_BUDGET_NS, 20_000_000)
    context.set_option(hmm.HMM_OPT_INJECT_SKIP_READY, 1)
    shape = hmm.make_shape(T, H, I, E, K, hmm.HMM_DTYPE_F32)
    ws = torch.empty(hmm.hmm_mx4_workspace_size(shape), dtype=torch.uint8, device=DEV)
    hmm.hmm_forward_mx4(context.handle, shape, x, ids, w, up.codes, up.scales, down.codes,
                        down.scales, torch.empty_like(x), ws)
    assert hmm.hmm_status(context.handle) == (hmm.HMM_ERR_TIMEOUT, hmm.HMM_STATUS_TIMEOUT)
    assert torch.equal(call(context, 1, x, ids, w, up, down), want)
