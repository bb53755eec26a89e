"""Microscaled 4-bit quantisation on the GPU against the 64-bit reference
(tests/mx4_ref.py): codes, scales and values are compared bit for bit."""
import numpy as np
import pytest
import torch

import dispatch_grouped_gemm_gb300 as hmm
from tests import mx4_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def draw(shape, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(shape, generator=g)
    v = v * torch.exp2(torch.randint(-12, 12, shape[:-1] + (1,), generator=g).float())
    return v.to(dtype)


def check(q, v):
    """q: Mx4Tensor of rows; v [N, K] float64 values in stored order."""
    codes, s = ref.quantize(v)
    packed, tiles = ref.store(codes, s)
    assert np.array_equal(q.scales.cpu().numpy(), tiles)
    got = q.codes.cpu().numpy()
    keep = np.repeat(s != 255, 16, -1)  # codes of NaN blocks are not defined
    assert got.shape == packed.shape and np.array_equal(got[keep], packed[keep])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,C", [(1, 8), (1, 32), (3, 40), (33, 128), (127, 136), (129, 264),
                                 (130, 1000), (5, 2056), (257, 96)])
def test_rows(R, C, dtype):
    v = draw((R, C), dtype, R + C)
    q = hmm.mx4_quantize(v.to(DEV))
    assert q.shape == (R, C)
    v64 = v.double().numpy()
    check(q, v64)
    for out in (torch.bfloat16, torch.float32):
        assert np.array_equal(q.dequantize(out).double().cpu().numpy(), ref.rounded(v64))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,K,N", [(1, 8, 8), (2, 40, 24), (3, 128, 64), (2, 136, 200),
                                   (1, 520, 136), (4, 64, 320)])
def test_experts(E, K, N, dtype):
    w = draw((E, N, K), dtype, E + K + N).transpose(1, 2).contiguous()
    q = hmm.mx4_quantize_experts(w.to(DEV))
    back = q.dequantize(dtype).double().cpu().numpy()
    for e in range(E):
        v = w[e].double().numpy().T
        check(hmm.Mx4Tensor.from_rows(q.codes[e], q.scales[e], K), v)
        assert np.array_equal(back[e], ref.rounded(v).T)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,K,I", [(1, 8, 8), (2, 40, 24), (3, 128, 64), (2, 264, 168), (1, 72, 40)])
def test_gate_up(E, K, I, dtype):
    w = draw((E, 2 * I, K), dtype, E + K + I).transpose(1, 2).contiguous()
    q = hmm.mx4_quantize_experts(w.to(DEV), gate_up=True)
    back = q.dequantize(dtype).double().cpu().numpy()
    for e in range(E):
        w64 = w[e].double().numpy()
        check(hmm.Mx4Tensor.from_rows(q.codes[e], q.scales[e], K), ref.gate_up_rows(w64))
        assert np.array_equal(back[e], ref.rounded(w64.T).T)


def test_every_bf16():
    """All 65536 bf16 bit patterns, one of them in each block."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = torch.zeros((65536, 32), dtype=torch.bfloat16)
    v[:, 5] = bits
    q = hmm.mx4_quantize(v.to(DEV))
    s = ref.scale_bytes(v.double().numpy())
    r = torch.arange(65536)
    got = q.scales.view(512, 512)[r // 128, r % 32 * 16 + r // 32 % 4 * 4].cpu().numpy()
    assert np.array_equal(got, s[:, 0])
    want = ref.rounded(v.double().numpy())
    got = q.dequantize(torch.float32).double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(np.nan_to_num(got), np.nan_to_num(want))


def test_ties_and_saturation():
    """Every sixteenth of the code range against the block's scale: ties to
    even, saturation from 6 up to the power of two."""
    m = torch.arange(-127, 128).float() / 16
    v = torch.zeros((255, 32))
    v[:, 0], v[:, 31] = 7.96875, m
    check(hmm.mx4_quantize(v.to(DEV)), v.double().numpy())


def test_extremes():
    tiny, big = 2.0 ** -149, torch.finfo(torch.float32).max
    rows = [[0.0], [tiny], [-tiny * 3], [big], [-big, 1.0], [2.0 ** -126], [2.0 ** -125, 2.0 ** -128],
            [float("inf"), 1.0], [float("nan"), 1.0], [-0.0]]
    v = torch.zeros((len(rows), 32))
    for i, r in enumerate(rows):
        v[i, :len(r)] = torch.tensor(r)
    q = hmm.mx4_quantize(v.to(DEV))
    check(q, v.double().numpy())
    got = q.dequantize(torch.float32).double().cpu().numpy()
    want = ref.rounded(v.double().numpy())
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.isnan(got).sum() == 64
    assert np.array_equal(np.nan_to_num(got), np.nan_to_num(want))


def test_strides_and_streams():
    wide = draw((50, 512), torch.bfloat16).to(DEV)
    for view in (wide[:, 8:272], wide[::2, :96], wide[:1, :64].expand(7, 64)):
        a, b = hmm.mx4_quantize(view), hmm.mx4_quantize(view.contiguous())
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    want = hmm.mx4_quantize(wide)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = hmm.mx4_quantize(wide)
        values = got.dequantize()
    s.synchronize()
    assert torch.equal(got.codes, want.codes) and torch.equal(values, want.dequantize())


def test_large_offsets():
    """More than 2^31 elements: rows far down, and the last expert of a stack."""
    x = torch.zeros(((1 << 31) // 4096 + 20000, 4096), dtype=torch.bfloat16, device=DEV)
    x[-130:] = draw((130, 4096), torch.bfloat16).to(DEV)
    q = hmm.mx4_quantize(x)
    assert torch.equal(q.dequantize()[-130:], hmm.mx4_quantize(x[-130:]).dequantize())
    w = x.view(-1)[: 33 * 4096 * 16384].view(33, 4096, 16384)
    w[-1] = draw((4096, 16384), torch.bfloat16).to(DEV)
    a = hmm.mx4_quantize_experts(w, gate_up=True)
    b = hmm.mx4_quantize_experts(w[-1:], gate_up=True)
    assert torch.equal(a.codes[-1:], b.codes) and torch.equal(a.scales[-1:], b.scales)
    assert torch.equal(a.dequantize()[-1:], b.dequantize())


def test_empty():
    q = hmm.mx4_quantize(torch.zeros((0, 64), device=DEV))
    assert q.shape == (0, 64) and q.dequantize().shape == (0, 64)


def test_refusals():
    x = torch.zeros((8, 64), device=DEV, dtype=torch.bfloat16)
    for bad, code in [(x[:, :60], -4), (x[:, 4:36], -4),
                      (torch.zeros((8, 36), device=DEV)[:, :32], -4)]:
        with pytest.raises(hmm.HmmError) as e:
            hmm.mx4_quantize(bad)
        assert e.value.code == code
    for bad in (x[0], x.t(), x.cpu()):
        with pytest.raises(ValueError):
            hmm.mx4_quantize(bad)
    with pytest.raises(TypeError):
        hmm.mx4_quantize(x.half())
    w = torch.zeros((2, 64, 24), device=DEV, dtype=torch.bfloat16)
    for bad, gate_up in [(torch.zeros((2, 60, 24), device=DEV), False),
                         (torch.zeros((2, 64, 12), device=DEV), False), (w, True)]:
        with pytest.raises(hmm.HmmError) as e:
            hmm.mx4_quantize_experts(bad, gate_up=gate_up)
        assert e.value.code == -4
    for bad in (x, w.transpose(1, 2), w.cpu()):
        with pytest.raises(ValueError):
            hmm.mx4_quantize_experts(bad)
    q = hmm.mx4_quantize(x)
    with pytest.raises(ValueError):
        hmm.Mx4Tensor.from_rows(q.codes, q.scales, 200)
    with pytest.raises(TypeError):
        hmm.Mx4Tensor.from_rows(q.codes.to(torch.int8), q.scales, 64)
    with pytest.raises(TypeError):
        q.dequantize(torch.float16)
