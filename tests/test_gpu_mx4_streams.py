"""4-bit expert products of several streams at once: calls that share the SMs
give the bits of calls made alone, and no wait between their tiles runs out."""
import pytest
import torch

import dispatch_grouped_gemm_gb300 as hmm
from tests.test_gpu_mx4_ffn import make

pytestmark = pytest.mark.gpu
DEV = "cuda"


def operands(*shape, seed):
    x, ids, w, W1, W2 = (t.to(DEV) for t in make(*shape, seed=seed))
    return (x, ids, w, hmm.mx4_quantize_experts(W1, gate_up=True), hmm.mx4_quantize_experts(W2))


# few tokens (every CTA's first tile counts), long batches, pairs of blocks
SHAPES = [(1, 2048, 1408, 16, 8), (64, 1024, 512, 32, 8), (1500, 2048, 1408, 16, 4),
          (2000, 2048, 2592, 2, 2)]


@pytest.mark.parametrize("a", range(len(SHAPES)))
@pytest.mark.parametrize("b", range(len(SHAPES)))
def test_two_streams_of_different_priority(a, b):
    """A tile belongs to a CTA that runs, so a call makes progress on whichever
    SMs the other call leaves to it."""
    calls = [operands(*SHAPES[a], seed=1), operands(*SHAPES[b], seed=2)]
    want = [hmm.moe_ffn_mx4(*c) for c in calls]
    torch.cuda.synchronize()
    low, high = torch.cuda.Stream(priority=0), torch.cuda.Stream(priority=-1)
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate((low, high)):
            with torch.cuda.stream(s):
                got[i].append(hmm.moe_ffn_mx4(*calls[i]))
    torch.cuda.synchronize()
    c = hmm.Context.for_device(torch.device(DEV, 0))
    assert hmm.hmm_status(c.handle) == (0, 0)
    for i in range(2):
        for y in got[i]:
            assert torch.equal(y, want[i])


def test_beside_a_kernel_that_holds_sms():
    """Matrix products of another stream, of higher priority, take SMs while the
    tiles run."""
    call = operands(2000, 2048, 2592, 2, 2, seed=3)
    want = hmm.moe_ffn_mx4(*call)
    m = torch.randn((2048, 2048), device=DEV).to(torch.bfloat16)
    torch.cuda.synchronize()
    s = torch.cuda.Stream(priority=-1)
    got = []
    for _ in range(10):
        with torch.cuda.stream(s):
            for _ in range(4):
                m @ m
        got.append(hmm.moe_ffn_mx4(*call))
    torch.cuda.synchronize()
    c = hmm.Context.for_device(torch.device(DEV, 0))
    assert hmm.hmm_status(c.handle) == (0, 0)
    for y in got:
        assert torch.equal(y, want)
