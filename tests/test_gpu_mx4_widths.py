"""Tiles of 128 and of 256 weight rows: on either side of the choice, which goes
by the token blocks, a token's result is the same bit for bit."""
import pytest
import torch

import dispatch_grouped_gemm_gb300 as hmm
from tests.test_gpu_mx4_ffn import make

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T,H,I,E,K", [(47, 3792, 536, 30, 4), (512, 4096, 1024, 8, 2),
                                       (700, 1024, 1024, 8, 2), (64, 1024, 512, 8, 2),
                                       (128, 2048, 1408, 8, 2)])
def test_widths_around_the_choice(T, H, I, E, K):
    x, ids, w, W1, W2 = (t.to(DEV) for t in make(T, H, I, E, K, seed=T))
    up, down = hmm.mx4_quantize_experts(W1, gate_up=True), hmm.mx4_quantize_experts(W2)
    got = [hmm.moe_ffn_mx4(x, ids, w, up, down) for _ in range(6)]
    one = torch.cat([hmm.moe_ffn_mx4(*(t.contiguous() for t in a), up, down)
                     for a in zip(x.split(8), ids.split(8), w.split(8))])
    for y in got:
        assert torch.equal(y, one)
