"""The open expert layer as it is used: the pieces together against the 64-bit formula,
streams, threads, graphs, and the update of the weights behind the gradients."""
import threading

import pytest
import torch

import dispatch_grouped_gemm_gb300 as hmm
from tests import open_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def layer(T=300, H=128, I=192, E=8, K=3, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(torch.bfloat16)

    x, up, down = normal(T, H), normal(E, H, I, std=H ** -0.5), normal(E, I, H, std=I ** -0.5)
    ids = torch.rand((T, E), generator=g, device=DEV).argsort(1)[:, :K].int().contiguous()
    w = torch.rand((T, K), generator=g, device=DEV)
    return x, ids, w, up, down, normal(T, H)


def forward(x, ids, w, up, down):
    """Experts with one matrix in and a squared ReLU."""
    r = hmm.moe_route(ids, up.shape[0])
    h = hmm.moe_grouped_mm(hmm.moe_dispatch(x, r), up, r.offsets)
    return hmm.moe_combine(hmm.moe_grouped_mm(torch.relu(h).square(), down, r.offsets), r, w)


def step(x, ids, w, up, down, dy):
    leaves = [t.detach().requires_grad_() for t in (x, w, up, down)]
    y = forward(leaves[0], ids, leaves[1], leaves[2], leaves[3])
    return (y.detach(),) + torch.autograd.grad(y, leaves, dy)


def exact(x, ids, w, up, down, dy):
    leaves = [t.detach().double().requires_grad_() for t in (x, w, up, down)]
    x, w, up, down = leaves
    y = torch.zeros_like(x)
    for e in range(up.shape[0]):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        o = torch.relu(x[t] @ up[e]).square() @ down[e]
        y = y.index_add(0, t, o * w[t, k].unsqueeze(1))
    return (y.detach(),) + torch.autograd.grad(y, leaves, dy.double())


def test_a_layer_and_its_gradients():
    """Against 64 bits.  On the way to each result are at most six roundings to bf16
    (2^-9 of a value on average at most, half a step 2^-8 / 2 .. of the relative norm:
    2^-9 each): h, its activation, the expert's row, and the same backwards; squaring
    doubles one of them.  Independent, their norms add to less than the sum, 8 * 2^-9."""
    args = layer()
    for name, got, want in zip(("y", "dx", "dw", "dup", "ddown"), step(*args), exact(*args)):
        assert got.shape == want.shape
        err = (got.double() - want).norm() / want.norm()
        assert err <= 8 * 2.0 ** -9, (name, err.item())


def test_in_place_of_the_fused_layer():
    """SwiGLU experts from the pieces: the fused layer's results up to roundings (each
    side rounds the hidden row, the expert's row and the sum, 2^-9 each, and the pieces
    the two halves of the first product too)."""
    x, ids, w, _, _, _ = layer(I=256)
    g = torch.Generator(device=DEV).manual_seed(5)
    up = (torch.randn((8, 128, 256), generator=g, device=DEV) * 128 ** -0.5).to(torch.bfloat16)
    down = (torch.randn((8, 128, 128), generator=g, device=DEV) * 128 ** -0.5).to(torch.bfloat16)
    want = hmm.moe_ffn(x, ids, w, up, down).double()
    r = hmm.moe_route(ids, 8)
    h = hmm.moe_grouped_mm(hmm.moe_dispatch(x, r), up, r.offsets)
    a = torch.nn.functional.silu(h[:, :128]) * h[:, 128:]
    got = hmm.moe_combine(hmm.moe_grouped_mm(a, down, r.offsets), r, w).double()
    assert (got - want).norm() <= 10 * 2.0 ** -9 * want.norm()


def test_first_call_of_a_thread():
    """A thread that has not used the device yet has no context of its own."""
    args = layer()
    want = step(*args)
    got = []

    def product():
        r = hmm.moe_route(args[1], 8)
        got.append(r)

    def other():
        o = torch.tensor([0, 100, 100, 200, 250, 260, 270, 280, 300], dtype=torch.int32)
        got.append(hmm.moe_grouped_mm(args[0], args[3], offsets))
        del o

    offsets = torch.tensor([0, 100, 100, 200, 250, 260, 270, 280, 300], dtype=torch.int32,
                           device=DEV)
    torch.cuda.synchronize()
    for f in (other, product):
        t = threading.Thread(target=f)
        t.start()
        t.join()
    assert len(got) == 2
    assert torch.equal(got[0], hmm.moe_grouped_mm(args[0], args[3], offsets))
    for a, b in zip(step(*args), want):
        assert torch.equal(a, b)


def test_streams():
    """Calls on two streams at once: each has its own buffers."""
    many = [layer(seed=s) for s in range(6)]
    want = [step(*a) for a in many]
    upd = [hmm.orthogonalize(w[3]) for w in want]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got, gupd = [], []
    for _ in range(4):
        got, gupd = [], []
        for i, a in enumerate(many):
            with torch.cuda.stream(streams[i % 3]):
                got.append(step(*a))
                gupd.append(hmm.orthogonalize(got[-1][3]))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for a, b in zip(g, w):
            assert torch.equal(a, b)
    for a, b in zip(gupd, upd):
        assert torch.equal(a, b)


def test_graph():
    """A whole step and the update behind it captured, replayed on changed inputs (other
    routings among them), two graphs in turn."""
    bufs = [torch.empty_like(t) for t in layer()]

    def both():
        out = step(*bufs)
        return out + tuple(hmm.orthogonalize(g) for g in out[3:])

    def fill(args):
        for b, a in zip(bufs, args):
            b.copy_(a)

    fill(layer())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = both()
        graphs.append((g, out))
    for seed in (3, 4, 5):
        args = layer(seed=seed)
        fill(args)
        for g, _ in graphs:
            g.replay()
        want = both()
        for _, out in graphs:
            for a, b in zip(out, want):
                assert torch.equal(a, b)


def test_update_of_stacked_weights():
    """What an optimiser does behind a step: momentum, orthogonalised, off the weights."""
    args = layer()
    _, _, _, dup, ddown = step(*args)
    for w, g in ((args[3], dup), (args[4], ddown)):
        m = torch.zeros_like(w).lerp_(g, 0.05)
        u = hmm.orthogonalize(m, scale=0.1)
        want = ref.orthogonalize(m, scale=0.1)
        # (test_gpu_orthogonalize has the derived bounds; half a percent is the claim)
        assert (u.double() - want).norm() <= 0.005 * want.norm()
        assert u.shape == w.shape and u.dtype == w.dtype
        w.sub_(u)
