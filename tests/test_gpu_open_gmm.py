"""Products grouped by expert (moe_grouped_mm) against the 64-bit formulas: forward and
both gradients, ragged and empty experts, one row to thousands, storage orders, strides,
rows of no expert, infinities behind a boundary."""
import pytest
import torch

import dispatch_grouped_gemm_gb300 as hmm
from tests import open_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"

# counts per expert, K, N: single rows; empty experts first, last and between; counts
# around the blocks (16, 64, 256) and K around the depth of a stage (64)
CASES = [
    ([1], 8, 8),
    ([0, 1, 0], 64, 256),
    ([3, 0, 5, 1], 72, 40),
    ([16, 17, 15, 1, 32, 33], 128, 264),
    ([64, 63, 65, 0, 128], 200, 512),
    ([255, 256, 257, 0, 0, 513], 256, 136),
    ([700], 1408, 320),
    ([5000, 3, 0, 40], 320, 776),
    ([1] * 70 + [0] * 20 + [2] * 30, 512, 512),
    # the rows of an expert in pieces: one hot expert between empty and small ones, whole
    # pieces, one row more and less
    ([0, 19000, 0, 5, 2049], 136, 264),
    ([2048, 4096, 2049, 6143, 10241, 1], 64, 128),
    ([20001], 72, 200),
]


def offsets_of(counts, head=0):
    o = [head]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32, device=DEV)


def problem(counts, K, N, dtype, layout="kn", tail=0, head=0, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    R, E = head + sum(counts) + tail, len(counts)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV).to(dtype)

    x, dy = normal(R, K), normal(R, N)
    w = normal(E, K, N) if layout == "kn" else normal(E, N, K).transpose(1, 2)
    return x, w, dy, offsets_of(counts, head)


# An fp32 accumulator: each MMA adds 16 products and the accumulator, 17 terms that are
# aligned to the largest and may lose up to 2^-23 of it each (twice that to be safe with
# the final normalisation): 17 * 2^-22 of the largest, which the sum of absolute values
# bounds, for every 16 of the depth.
PER_MMA = 17 * 2.0 ** -22


def check(x, w, dy, o, y, dx, dw):
    counts = (o[1:] - o[:-1]).tolist()
    K, N = w.shape[1:]
    x, w, dy = x.detach(), w.detach(), dy.detach()
    wt = w.transpose(1, 2)
    ref.assert_close("y", y, ref.grouped_mm(x, w, o),
                     ref.grouped_mm(x.abs(), w.abs(), o) * ((K + 15) // 16) * PER_MMA)
    if dx is not None:
        ref.assert_close("dx", dx, ref.grouped_mm(dy, wt, o),
                         ref.grouped_mm(dy.abs(), wt.abs(), o) * ((N + 15) // 16) * PER_MMA)
    if dw is not None:
        steps = torch.tensor([(c + 15) // 16 for c in counts], device=DEV).view(-1, 1, 1)
        ref.assert_close("dw", dw, ref.grouped_mm_dw(x, dy, o),
                         ref.grouped_mm_dw(x.abs(), dy.abs(), o) * steps * PER_MMA)


def run(x, w, dy, o):
    x, w = x.detach().requires_grad_(), w.detach().requires_grad_()
    y = hmm.moe_grouped_mm(x, w, o)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    return y.detach(), dx, dw


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", CASES)
def test_forward(case, dtype, layout):
    x, w, dy, o = problem(*case, dtype, layout)
    check(x, w, dy, o, hmm.moe_grouped_mm(x, w, o), None, None)


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", CASES)
def test_gradients(case, dtype, layout):
    x, w, dy, o = problem(*case, dtype, layout)
    y, dx, dw = run(x, w, dy, o)
    assert dw.shape == w.shape
    check(x, w, dy, o, y, dx, dw)


@pytest.mark.parametrize("count", list(range(1, 35)) + [47, 48, 49, 95, 96, 97, 127, 129, 143, 144,
                                                        145, 239, 241])
def test_every_block_height(count):
    """Every number of 16-row steps that a block can have, beside a neighbour."""
    x, w, dy, o = problem([count, 7], 64, 64, torch.bfloat16)
    check(x, w, dy, o, *run(x, w, dy, o))


@pytest.mark.parametrize("head,tail", [(0, 1), (0, 77), (5, 0), (3, 300)])
def test_rows_of_no_expert(head, tail):
    """They are zeros in y and dx and add nothing to dw, whatever they hold."""
    counts = [9, 0, 130]
    x, w, dy, o = problem(counts, 96, 160, torch.bfloat16, head=head, tail=tail)
    n = head + sum(counts)
    clean_x, clean_dy = x.clone(), dy.clone()
    for t, c in ((x, clean_x), (dy, clean_dy)):
        t[:head], t[n:] = float("nan"), float("inf")
        c[:head], c[n:] = 0, 0
    y, dx, dw = run(x, w, dy, o)
    for t in (y, dx):
        assert not bool(t[:head].any()) and not bool(t[n:].any())
    check(clean_x, w, clean_dy, o, y, dx, dw)


def test_neighbours_do_not_mix():
    """Infinities and NaN of one expert's rows or weights stay in its results."""
    counts = [5, 70, 6, 64, 1]
    x, w, dy, o = problem(counts, 128, 128, torch.bfloat16)
    bad = slice(int(o[1]), int(o[2]))
    clean = run(x, w, dy, o)
    x[bad], dy[bad] = float("nan"), float("inf")
    w[1] = float("nan")
    y, dx, dw = run(x, w, dy, o)
    keep = torch.ones(x.shape[0], dtype=torch.bool, device=DEV)
    keep[bad] = False
    assert torch.equal(y[keep], clean[0][keep]) and torch.equal(dx[keep], clean[1][keep])
    for e in (0, 2, 3, 4):
        assert torch.equal(dw[e], clean[2][e])
    assert bool(torch.isnan(y[bad]).all()) and not bool(torch.isfinite(dw[1]).any())


def test_empty():
    w = torch.randn((3, 64, 32), device=DEV).to(torch.bfloat16)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    y, dx, dw = run(x, w, torch.empty((0, 32), dtype=torch.bfloat16, device=DEV),
                    offsets_of([0, 0, 0]))
    assert y.shape == (0, 32) and dx.shape == (0, 64) and not bool(dw.any())
    x = torch.randn((7, 64), device=DEV).to(torch.bfloat16)  # rows, but none of an expert
    y, dx, dw = run(x, w, torch.ones((7, 32), dtype=torch.bfloat16, device=DEV),
                    offsets_of([0, 0, 0]))
    assert not bool(y.any()) and not bool(dx.any()) and not bool(dw.any())


def test_strides():
    """Rows apart, operands off 16 bytes, broadcast rows, columns without unit stride,
    weights that are slices or one matrix for all experts: copied where TMA needs it."""
    counts, K, N = [20, 33, 0, 4], 128, 64
    R, E = sum(counts), 4
    o = offsets_of(counts)
    g = torch.Generator(device=DEV).manual_seed(1)
    big = torch.randn((R, 3 * K + 8), generator=g, device=DEV).to(torch.bfloat16)
    bigw = torch.randn((E, K + 3, 2 * N + 8), generator=g, device=DEV).to(torch.bfloat16)
    bigdy = torch.randn((R, 2 * N + 4), generator=g, device=DEV).to(torch.bfloat16)
    xs = (big[:, :K], big[:, 8:K + 8], big[:, 3:K + 3], big[:, ::3][:, :K], big[0, :K].expand(R, K))
    ws = (bigw[:, :K, :N], bigw[:, 3:, 8:N + 8], bigw[:, :K, 1:N + 1],
          bigw[:1, :K, :N].expand(E, K, N), bigw[:, :N, :K].transpose(1, 2))
    for x in xs:
        for w in ws:
            for dy in (bigdy[:, :N], bigdy[:, 1:N + 1], bigdy[0, :N].expand(R, N)):
                got = run(x, w, dy, o)
                want = run(*(t.clone(memory_format=torch.contiguous_format) for t in (x, w, dy)), o)
                for a, b in zip(got, want):
                    assert torch.equal(a, b)
    w1 = torch.randn((1, K, N), generator=g, device=DEV).to(torch.bfloat16).requires_grad_()
    y = hmm.moe_grouped_mm(xs[0], w1.expand(E, K, N), o)
    (dw,) = torch.autograd.grad(y, w1, torch.ones_like(y))
    ones = torch.ones((R, N), dtype=torch.bfloat16, device=DEV)
    want = ref.grouped_mm_dw(xs[0], ones, offsets_of([R]))
    # E rounded gradients, summed and rounded again
    mass = ref.grouped_mm_dw(xs[0].abs(), ones, offsets_of([R]))
    ref.assert_close("dw", dw, want, mass * E * 2.0 ** -8)


@pytest.mark.parametrize("offsets", [[0, 50, 20, 64], [-7, 10, 30, 64], [0, 10, 30, 900],
                                     [70, 80, 90, 100], [64, 0, 64, 0]])
def test_unordered_offsets_stay_inside(offsets):
    """Results are unspecified, but nothing outside the arrays is touched."""
    x, w, dy, _ = problem([64, 0, 0], 64, 64, torch.bfloat16)
    o = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    guard = torch.full((3, 64, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    out = guard[1]
    d = hmm.make_gmm(64, 64, 64, 3)
    h = hmm.Context.for_device(x.device).handle
    hmm.hmm_grouped_mm(h, d, x, w, o, out)
    hmm.hmm_grouped_mm_dx(h, d, dy, w, o, out)
    run(x, w, dy, o)
    assert hmm.hmm_status(h) == (0, 0)
    assert bool((guard[0] == 7).all()) and bool((guard[2] == 7).all())


@pytest.mark.parametrize("offsets", [[0, 19000, 0, 19000, 0, 19000],
                                     [19000, 0, 19000, 0, 19000, 10],
                                     [-7, 8000, 3000, 40000, 6000, 19000]])
def test_unordered_offsets_stay_in_the_workspace(offsets):
    """The pieces of an expert's rows have places in the workspace that sums of rows
    bound: with offsets out of order too."""
    R, K, N, E = 19000, 64, 64, 5
    x, _, dy, _ = problem([R, 0, 0, 0, 0], K, N, torch.bfloat16)
    o = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    d = hmm.make_gmm(R, K, N, E)
    size = hmm.hmm_grouped_mm_workspace_size(d)
    assert size > 0
    guard = torch.full((size + 65536,), 7, dtype=torch.uint8, device=DEV)
    dw = torch.empty((E, K, N), dtype=torch.bfloat16, device=DEV)
    h = hmm.Context.for_device(x.device).handle
    hmm.hmm_grouped_mm_dw(h, d, x, dy, o, dw, guard[:size])
    assert hmm.hmm_status(h) == (0, 0)
    assert bool((guard[size:] == 7).all())


def test_only_the_gradients_asked_for():
    x, w, dy, o = problem([20, 5], 64, 64, torch.bfloat16)
    full = run(x, w, dy, o)
    y = hmm.moe_grouped_mm(x.requires_grad_(), w, o)
    assert torch.equal(torch.autograd.grad(y, x, dy)[0], full[1])
    y = hmm.moe_grouped_mm(x.detach(), w.requires_grad_(), o)
    assert torch.equal(torch.autograd.grad(y, w, dy)[0], full[2])
    with pytest.raises(RuntimeError, match="no second derivative"):
        y = hmm.moe_grouped_mm(x.detach(), w, o)
        (dw,) = torch.autograd.grad(y.square().sum(), w, create_graph=True)
        dw.sum().backward()


def test_many_tiles():
    """More tiles than pairs of SMs in each direction, weights of several hundred MB."""
    x, w, dy, o = problem([900, 0, 411, 1300, 77, 5], 2048, 2816, torch.bfloat16)
    check(x, w, dy, o, *run(x, w, dy, o))


def test_results_repeat():
    x, w, dy, o = problem([900, 0, 411, 1300, 77, 5], 512, 768, torch.bfloat16)
    a, b = run(x, w, dy, o), run(x, w, dy, o)
    for s, t in zip(a, b):
        assert torch.equal(s, t)
