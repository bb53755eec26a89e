"""The combine of few tokens (every row loaded before the first is added) and of
more: the same bits on either side of the choice, which goes by T, H and K."""
import pytest
import torch

import dispatch_grouped_gemm_gb300 as hmm
from tests.test_gpu_mx4_ffn import make

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T,H,I,E,K", [(300, 4096, 64, 16, 8), (256, 4096, 64, 16, 8),
                                       (600, 512, 32, 4, 2), (1000, 768, 32, 9, 5),
                                       (140, 2056, 32, 3, 1)])
def test_combine_around_the_choice(T, H, I, E, K):
    x, ids, w, W1, W2 = (t.to(DEV) for t in make(T, H, I, E, K, seed=T))
    up, down = hmm.mx4_quantize_experts(W1, gate_up=True), hmm.mx4_quantize_experts(W2)
    ids[7, K - 1] = E  # skipped: a slot without a row
    def parts(f, n):
        return torch.cat([f(*(t.contiguous() for t in a))
                          for a in zip(x.split(n), ids.split(n), w.split(n))])
    for f in (lambda x, i, w: hmm.moe_ffn(x, i, w, W1, W2),
              lambda x, i, w: hmm.moe_ffn_mx4(x, i, w, up, down)):
        assert torch.equal(f(x, ids, w), parts(f, 20))
    c = hmm.Context.for_device(torch.device(DEV, 0))
    assert hmm.hmm_status(c.handle)[1] == hmm.HMM_STATUS_EXPERT_ID  # and cleared
