"""Argument checks of the open layer and of the orthogonalised update, on the CPU: codes
of the C entries (every check precedes device work), refusals of the torch layer, and the
device and stream that a call goes to, on stand-ins for tensors."""
import ctypes
import types

import pytest
import torch

import dispatch_grouped_gemm_gb300 as hmm
from dispatch_grouped_gemm_gb300 import build as hbuild
from tests.test_devices import Fake

BAD_ARG, BAD_SHAPE, BAD_DTYPE, BAD_LAYOUT = (
    hmm._C[n] for n in ("HMM_ERR_ARG", "HMM_ERR_SHAPE", "HMM_ERR_DTYPE", "HMM_ERR_LAYOUT"))
F16, BF16, F32 = hmm.HMM_DTYPE_F16, hmm.HMM_DTYPE_BF16, hmm.HMM_DTYPE_F32
MUON = (hmm.MUON_COEFFICIENTS,) * 5


@pytest.fixture(scope="module")
def lib():
    hbuild.build()
    return hmm.load_library()


def code(call, *args, **kw):
    if not call.__name__.endswith("_size"):
        kw["stream"] = 0
    with pytest.raises(hmm.HmmError) as e:
        call(*args, **kw)
    return e.value.code


@pytest.mark.parametrize("kw,want", [
    (dict(R=-1), BAD_SHAPE), (dict(R=2 ** 31 - 1), BAD_SHAPE), (dict(K=0), BAD_SHAPE),
    (dict(N=-8), BAD_SHAPE), (dict(E=0), BAD_SHAPE), (dict(E=1025), BAD_SHAPE),
    (dict(K=2 ** 20 + 8), BAD_SHAPE), (dict(K=60), BAD_LAYOUT), (dict(N=4), BAD_LAYOUT),
    (dict(ld_x=56), BAD_SHAPE), (dict(ld_x=68), BAD_LAYOUT), (dict(ld_dy=120), BAD_SHAPE),
    (dict(ld_dy=132), BAD_LAYOUT), (dict(ld_w=120), BAD_SHAPE), (dict(ld_w=129), BAD_SHAPE),
    (dict(ld_w=132, stride_w=2 ** 20), BAD_LAYOUT), (dict(stride_w=64), BAD_SHAPE),
    (dict(stride_w=-8), BAD_SHAPE), (dict(stride_w=64 * 128 + 4), BAD_LAYOUT),
    (dict(ld_x=2 ** 38, R=2 ** 20), BAD_SHAPE), (dict(dtype=F32), BAD_DTYPE),
    (dict(dtype=9), BAD_DTYPE), (dict(w_layout=2), BAD_ARG),
])
def test_grouped_product_descriptors(lib, kw, want):
    d = dict(R=100, K=64, N=128, E=4)
    d.update(kw)
    assert code(hmm.hmm_grouped_mm_workspace_size, hmm.make_gmm(**d)) == want


def test_grouped_product_workspace(lib):
    """Whole experts need none; pieces never more places than twice the rows' whole
    pieces, whatever the experts' rows."""
    size = hmm.hmm_grouped_mm_workspace_size
    assert size(hmm.make_gmm(0, 64, 64, 1)) == 0
    assert size(hmm.make_gmm(4096, 64, 64, 1)) == 0
    assert size(hmm.make_gmm(131072, 2048, 7168, 32)) == 0
    for R, K, N, E in ((65536, 256, 256, 1), (131071, 512, 1024, 8), (2 ** 30, 64, 64, 1)):
        n = size(hmm.make_gmm(R, K, N, E))
        assert n > 0 and n % 16 == 0
        assert n == size(hmm.make_gmm(R, N, K, E, w_layout=hmm.HMM_W_NK))
        assert (n - 4112) // (K * N * 4) <= 2 * (R // 2048)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), BAD_SHAPE), (dict(H=0), BAD_SHAPE), (dict(K=0), BAD_SHAPE),
    (dict(K=33), BAD_SHAPE), (dict(E=0), BAD_SHAPE), (dict(E=1025), BAD_SHAPE), (dict(ld=99), BAD_SHAPE),
    (dict(H=2 ** 20 + 1), BAD_SHAPE), (dict(T=2 ** 30), BAD_SHAPE), (dict(dtype=7), BAD_DTYPE),
    (dict(weights_dtype=F16), BAD_DTYPE),
])
def test_row_descriptors(lib, kw, want):
    d = dict(T=5, H=100, K=2, E=4)
    d.update(kw)
    d = hmm.make_rows(**d)
    handle = ctypes.c_void_p(64)  # (not looked into before the descriptor is checked)
    assert code(hmm.hmm_dispatch, handle, d, 64, 64, 64, 64) == want
    assert code(hmm.hmm_dispatch_grad, handle, d, 64, 64, 64) == want
    assert code(hmm.hmm_combine, handle, d, 64, 64, 64, 64) == want
    assert code(hmm.hmm_combine_grad, handle, d, 64, 64, 64, 64, 64, 64, 64) == want


def test_pointers(lib):
    """None of them NULL, element aligned (rows) or 16-byte aligned (products)."""
    handle = ctypes.c_void_p(64)
    rows, gmm = hmm.make_rows(5, 100, 2, 4), hmm.make_gmm(100, 64, 64, 4)
    pieces = hmm.make_gmm(65536, 64, 64, 1)
    ortho = hmm.make_ortho(2, 16, 16, MUON)
    for call, d, n, misaligned in (
            (hmm.hmm_dispatch, rows, 4, 65), (hmm.hmm_dispatch_grad, rows, 3, 65),
            (hmm.hmm_combine, rows, 4, 65), (hmm.hmm_grouped_mm, gmm, 4, 66),
            (hmm.hmm_grouped_mm_dx, gmm, 4, 66), (hmm.hmm_grouped_mm_dw, gmm, 4, 66)):
        assert code(call, None, d, *[64] * n) == BAD_ARG
        for i in range(n):
            args = [64] * n
            args[i] = None
            assert code(call, handle, d, *args) == BAD_ARG
            args[i] = misaligned
            assert code(call, handle, d, *args) == BAD_LAYOUT
    # without d_topk_weights the rows are not read
    assert code(hmm.hmm_combine_grad, handle, rows, None, 64, 64, 64, 64, 64, 64) == BAD_ARG
    assert code(hmm.hmm_combine_grad, handle, rows, 64, 64, 64, 64, 65, 64, 64) == BAD_LAYOUT
    # nothing asked for
    hmm.hmm_combine_grad(handle, rows, 64, 64, 64, 64, 64, None, None, stream=0)
    # the workspace of pieces
    assert code(hmm.hmm_grouped_mm_dw, handle, pieces, 64, 64, 64, 64) == BAD_ARG
    short = torch.empty(64, dtype=torch.uint8)
    assert code(hmm.hmm_grouped_mm_dw, handle, pieces, 64, 64, 64, 64,
                short) == hmm._C["HMM_ERR_CAPACITY"]
    assert code(hmm.hmm_orthogonalize, handle, ortho, 64, 64, None) == BAD_ARG
    assert code(hmm.hmm_orthogonalize, handle, ortho, 65, 64, short) == BAD_LAYOUT
    assert code(hmm.hmm_orthogonalize, handle, ortho, 64, 64,
                short) == hmm._C["HMM_ERR_CAPACITY"]


def test_calls_without_rows_do_nothing(lib):
    """(No device is touched: there may be none.)"""
    handle = ctypes.c_void_p(64)
    rows, gmm = hmm.make_rows(0, 100, 2, 4), hmm.make_gmm(0, 64, 64, 4)
    hmm.hmm_dispatch(handle, rows, None, None, None, None, stream=0)
    hmm.hmm_dispatch_grad(handle, rows, None, None, None, stream=0)
    hmm.hmm_combine(handle, rows, None, None, None, None, stream=0)
    hmm.hmm_combine_grad(handle, rows, None, None, None, None, None, None, None, stream=0)
    hmm.hmm_grouped_mm(handle, gmm, None, None, None, None, stream=0)
    hmm.hmm_grouped_mm_dx(handle, gmm, None, None, None, None, stream=0)
    hmm.hmm_orthogonalize(handle, hmm.make_ortho(0, 16, 16, MUON), None, None, None, stream=0)


@pytest.mark.parametrize("kw,want", [
    (dict(batch=-1), BAD_SHAPE), (dict(batch=65536), BAD_SHAPE), (dict(M=0), BAD_SHAPE),
    (dict(N=2 ** 17 + 1), BAD_SHAPE), (dict(ld=15), BAD_SHAPE), (dict(stride=-1), BAD_SHAPE),
    (dict(dtype=9), BAD_DTYPE), (dict(out_dtype=F32), BAD_DTYPE),
    (dict(coefficients=()), BAD_ARG), (dict(coefficients=MUON[:1] * 33), BAD_ARG),
    (dict(eps=-1.0), BAD_ARG), (dict(eps=float("nan")), BAD_ARG), (dict(eps=float("inf")), BAD_ARG),
    (dict(scale=float("inf")), BAD_ARG), (dict(scale=float("nan")), BAD_ARG),
    (dict(coefficients=((float("nan"), 0.0, 0.0),)), BAD_ARG),
    (dict(coefficients=((3e6, 0.0, 0.0),)), BAD_ARG),
    # singular values that grow past 2^20
    (dict(coefficients=((1000.0, 0.0, 0.0),) * 3), BAD_ARG),
    (dict(batch=65535, M=2 ** 15, N=2 ** 15), BAD_SHAPE),
])
def test_update_descriptors(lib, kw, want):
    d = dict(batch=2, M=16, N=16, coefficients=MUON)
    d.update(kw)
    assert code(hmm.hmm_orthogonalize_workspace_size, hmm.make_ortho(**d)) == want


def test_update_workspace_grows_with_the_stack(lib):
    def size(batch, M, N):
        return hmm.hmm_orthogonalize_workspace_size(hmm.make_ortho(batch, M, N, MUON))

    # two X in 22 bits and A, B in 16 are its bulk; both orientations cost the same
    assert size(4, 1024, 512) == size(4, 512, 1024)
    assert size(8, 512, 1024) >= 2 * 8 * (4 * 512 * 1024 // 2 + 2 * 512 * 512)
    assert size(1, 1, 1) > 0 and size(2, 512, 512) < size(3, 512, 512)


# ------------------------------------------------------------------ torch layer
class Stand(Fake):
    """A stand-in that can be cut and copied."""

    layout = torch.strided

    def split(self, sizes):
        return [Stand((n,), self.dtype, self.index) for n in sizes]

    def view(self, *shape):
        return Stand(shape, self.dtype, self.index)

    def reshape(self, *shape):
        return Stand(tuple(self.numel() // (self.shape[-1] * self.shape[-2]) if n == -1 else n
                           for n in shape), self.dtype, self.index)

    def numel(self):
        return self.shape.numel()

    def contiguous(self):
        return self

    def detach(self):
        return self


@pytest.fixture
def calls(monkeypatch):
    """(function name, stream) of every call of the library: streams are 1000 +
    device, device 0 is current."""
    got = []

    class Library:
        def __getattr__(self, name):
            def call(*args):
                if not name.endswith("_size"):
                    got.append((name, args[-1]))
                return 0
            return call

    def empty(shape, dtype=None, device=None):
        shape = (shape,) if isinstance(shape, int) else shape
        return Stand(shape, dtype, torch.device(device).index)

    monkeypatch.setattr(hmm, "load_library", lambda lib=Library(): lib)
    monkeypatch.setattr(hmm, "_raw_stream", lambda index: 1000 + index)
    monkeypatch.setattr(hmm, "_current_device", lambda: 0)
    monkeypatch.setattr(hmm, "_route_call", lambda T, E, K: (hmm.HmmShape(), 16))
    monkeypatch.setattr(hmm, "_gmm_workspace", lambda R, K, N, E: 16)
    monkeypatch.setattr(hmm, "_ortho_call", lambda *a: (hmm.make_ortho(1, 8, 8, MUON), 16))
    monkeypatch.setattr(hmm.Context, "for_device", classmethod(
        lambda cls, device: types.SimpleNamespace(handle=ctypes.c_void_p(1))))
    monkeypatch.setattr(hmm.torch, "empty", empty)
    monkeypatch.setattr(hmm.torch, "empty_like", lambda t: empty(t.shape, t.dtype, t.device))
    return got


def stand(*shape, dtype=torch.bfloat16, index=0):
    return Stand(shape, dtype, index)


def ints(*shape, index=0):
    return Stand(shape, torch.int32, index)


def routing(index=0, T=6, K=2, E=4):
    return hmm.MoeRouting(ints(E, index=index), ints(E + 1, index=index), ints(T, K, index=index),
                          ints(T * K, index=index))


@pytest.mark.parametrize("index", [0, 1])
def test_calls_go_to_a_stream_of_their_tensors_device(calls, index):
    r = hmm.moe_route(ints(6, 2, index=index), 4)
    x, rows, w = (stand(*shape, index=index) for shape in ((6, 16), (12, 16), (4, 16, 24)))
    weights = stand(6, 2, dtype=torch.float32, index=index)
    assert hmm.moe_dispatch(x, r).shape == (12, 16)
    assert hmm.moe_grouped_mm(rows, w, r.offsets).shape == (12, 24)
    assert hmm.moe_combine(rows, r, weights).device.index == index
    assert hmm.orthogonalize(w).dtype == torch.bfloat16
    stream = 1000 + index
    assert calls == [(n, stream) for n in ("hmm_route", "hmm_dispatch", "hmm_grouped_mm",
                                           "hmm_combine", "hmm_orthogonalize")]
    calls.clear()
    with torch.no_grad():  # as autograd calls them without create_graph
        ctx = types.SimpleNamespace(saved_tensors=(x, r.slot2row), routing=r)
        hmm._Dispatch.backward(ctx, rows)
        ctx = types.SimpleNamespace(saved_tensors=(rows, weights, r.slot2row, r.offsets),
                                    routing=r, needs_input_grad=(True, False, True))
        hmm._Combine.backward(ctx, x)
        ctx = types.SimpleNamespace(saved_tensors=(rows, w, r.offsets),
                                    needs_input_grad=(True, True, False))
        hmm._GroupedMM.backward(ctx, stand(12, 24, index=index))
    assert calls == [(n, stream) for n in ("hmm_dispatch_grad", "hmm_combine_grad",
                                           "hmm_grouped_mm_dx", "hmm_grouped_mm_dw")]


def test_operands_of_two_devices_are_refused(calls):
    r, x, rows, w = routing(), stand(6, 16), stand(12, 16), stand(4, 16, 24)
    weights = stand(6, 2, dtype=torch.float32)
    with pytest.raises(ValueError, match="device"):
        hmm.MoeRouting(ints(4), ints(5), ints(6, 2, index=1), ints(12))
    for call in (lambda: hmm.moe_dispatch(stand(6, 16, index=1), r),
                 lambda: hmm.moe_combine(stand(12, 16, index=1), r, weights),
                 lambda: hmm.moe_combine(rows, r, stand(6, 2, dtype=torch.float32, index=1)),
                 lambda: hmm.moe_combine(rows, routing(1), weights),
                 lambda: hmm.moe_grouped_mm(rows, stand(4, 16, 24, index=1), r.offsets),
                 lambda: hmm.moe_grouped_mm(rows, w, ints(5, index=1)),
                 lambda: hmm.moe_dispatch(x, routing(1))):
        with pytest.raises(ValueError, match="device"):
            call()
    assert not calls


def test_refused_arguments(calls):
    r, rows, w = routing(), stand(12, 16), stand(4, 16, 24)
    weights = stand(6, 2, dtype=torch.float32)
    f64, i64 = torch.float64, torch.int64
    wrong = [
        (TypeError, hmm.moe_route, stand(6, 2, dtype=i64), 4),
        (ValueError, hmm.moe_route, ints(12), 4),
        (ValueError, hmm.MoeRouting, ints(4), ints(4), ints(6, 2), ints(12)),
        (ValueError, hmm.MoeRouting, ints(4), ints(5), ints(6, 2), ints(11)),
        (ValueError, hmm.MoeRouting, ints(4), ints(5), ints(12), ints(12)),
        (TypeError, hmm.MoeRouting, ints(4), ints(5), stand(6, 2, dtype=i64), ints(12)),
        (ValueError, hmm.moe_dispatch, stand(5, 16), r),
        (ValueError, hmm.moe_dispatch, stand(6, 2, 8), r),
        (TypeError, hmm.moe_dispatch, stand(6, 16, dtype=f64), r),
        (ValueError, hmm.moe_combine, stand(11, 16), r, weights),
        (ValueError, hmm.moe_combine, rows, r, stand(6, 3, dtype=torch.float32)),
        (TypeError, hmm.moe_combine, stand(12, 16, dtype=f64), r, weights),
        (TypeError, hmm.moe_combine, rows, r, stand(6, 2, dtype=torch.float16)),
        (ValueError, hmm.moe_grouped_mm, rows, stand(4, 24, 16), ints(5)),
        (ValueError, hmm.moe_grouped_mm, rows, w, ints(4)),
        (ValueError, hmm.moe_grouped_mm, rows, stand(16, 24), ints(5)),
        (ValueError, hmm.moe_grouped_mm, stand(12, 12), stand(4, 12, 24), ints(5)),
        (ValueError, hmm.moe_grouped_mm, stand(12, 0), stand(4, 0, 24), ints(5)),
        (TypeError, hmm.moe_grouped_mm, stand(12, 16, dtype=torch.float16), w, ints(5)),
        (TypeError, hmm.moe_grouped_mm, stand(12, 16, dtype=torch.float32),
         stand(4, 16, 24, dtype=torch.float32), ints(5)),
        (TypeError, hmm.moe_grouped_mm, rows, w, stand(5, dtype=i64)),
        (ValueError, hmm.orthogonalize, stand(16)),
        (TypeError, hmm.orthogonalize, stand(16, 16, dtype=f64)),
    ]
    for error, call, *args in wrong:
        with pytest.raises(error):
            call(*args)
    g = stand(4, 16, 24)
    for error, kw in ((TypeError, dict(out_dtype=torch.float32)),
                      (ValueError, dict(steps=4, coefficients=MUON)),
                      (ValueError, dict(steps=0, coefficients=())),
                      (ValueError, dict(coefficients=(1.0, 2.0))),
                      (ValueError, dict(steps=1, coefficients=((1.0, 2.0),)))):
        with pytest.raises(error):
            hmm.orthogonalize(g, **kw)
    g.requires_grad = True
    with pytest.raises(RuntimeError, match="no backward"):
        hmm.orthogonalize(g)
    assert not calls


def test_host_tensors_are_refused():
    x, w = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(2, 16, 16, dtype=torch.bfloat16)
    for call in (lambda: hmm.moe_route(torch.zeros(4, 2, dtype=torch.int32), 4),
                 lambda: hmm.moe_grouped_mm(x, w, torch.zeros(3, dtype=torch.int32)),
                 lambda: hmm.orthogonalize(w)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
