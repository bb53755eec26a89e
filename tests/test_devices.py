"""The torch layer of the router and the 4-bit experts in a process with several
devices, on stand-ins for tensors (no GPU): operands of different devices are
refused before any device work, and a call goes to the current stream of its
tensors' device, whichever device is current."""
import ctypes
import types

import pytest
import torch

import dispatch_grouped_gemm_gb300 as hmm


class Fake:
    """What the torch layer looks at of a tensor on CUDA device `index`."""

    is_cuda, requires_grad = True, False

    def __init__(self, shape, dtype, index):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, index
        self.device = torch.device("cuda", index)

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def stride(self, i):
        n = 1
        for s in self.shape[i + 1:]:
            n *= s
        return n

    def data_ptr(self):
        return 4096


@pytest.fixture
def calls(monkeypatch):
    """(function name, stream) of every call of the library: streams are 1000 +
    device, device 0 is current."""
    got = []

    class Library:
        def __getattr__(self, name):
            def call(*args):
                got.append((name, args[-1]))
                return 0
            return call

    def fake(shape, dtype=None, device=None):
        shape = (shape,) if isinstance(shape, int) else shape
        return Fake(shape, dtype, torch.device(device).index)

    monkeypatch.setattr(hmm, "load_library", lambda lib=Library(): lib)
    monkeypatch.setattr(hmm, "_raw_stream", lambda index: 1000 + index)
    monkeypatch.setattr(hmm, "_current_device", lambda: 0)
    monkeypatch.setattr(hmm, "_mx4_call",
                        lambda T, H, I, E, K, w: (hmm.HmmShape(T, H, I, E, K, w, 0), 256))
    monkeypatch.setattr(hmm.Context, "for_device", classmethod(
        lambda cls, device: types.SimpleNamespace(handle=ctypes.c_void_p(1))))
    monkeypatch.setattr(hmm.torch, "empty", fake)
    return got


def ffn_arguments(index):
    def stack(layout, stored, rows, cols):
        return hmm.Mx4Tensor(Fake((4, stored, cols // 2), torch.uint8, index),
                             Fake((4, 1, 1, 512), torch.uint8, index), 4, rows, cols, layout)

    return [Fake((3, 64), torch.bfloat16, index), Fake((3, 2), torch.int32, index),
            Fake((3, 2), torch.float32, index), stack(hmm.HMM_MX4_GATE_UP, 64, 64, 64),
            stack(hmm.HMM_MX4_COLUMNS, 64, 64, 32)]


def test_operands_of_two_devices_are_refused(calls):
    other = ffn_arguments(1)
    for i in range(5):
        mixed = ffn_arguments(0)
        mixed[i] = other[i]
        with pytest.raises(ValueError, match="device"):
            hmm.moe_ffn_mx4(*mixed)
    scales_elsewhere = ffn_arguments(0)
    scales_elsewhere[4].scales = other[4].scales
    with pytest.raises(ValueError, match="device"):
        hmm.moe_ffn_mx4(*scales_elsewhere)
    assert not calls


@pytest.mark.parametrize("index", [0, 1])
def test_calls_go_to_a_stream_of_their_tensors_device(calls, index):
    y = hmm.moe_ffn_mx4(*ffn_arguments(index))
    assert y.device.index == index
    hmm.moe_gate(Fake((3, 32), torch.float32, index), 4)
    q = hmm.mx4_quantize(Fake((3, 64), torch.bfloat16, index))
    q.dequantize()
    hmm.mx4_quantize_experts(Fake((4, 64, 64), torch.bfloat16, index))
    assert calls == [(name, 1000 + index) for name in (
        "hmm_forward_mx4", "hmm_gate_forward", "hmm_mx4_quantize", "hmm_mx4_dequantize",
        "hmm_mx4_quantize")]
    calls.clear()
    saved = (Fake((3, 32), torch.float32, index), Fake((3, 4), torch.int32, index))
    ctx = types.SimpleNamespace(saved_tensors=saved, gate=hmm.make_gate(3, 32, 4))
    with torch.no_grad():  # as autograd calls it without create_graph
        hmm._MoEGate.backward(ctx, None, Fake((3, 4), torch.float32, index), None)
    assert calls == [("hmm_gate_backward", 1000 + index)]
