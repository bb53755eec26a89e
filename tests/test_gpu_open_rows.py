"""Rows into expert order and back (moe_route, moe_dispatch, moe_combine) against the
64-bit formulas: forward, gradients, invalid ids, strides, odd sizes, empty batches."""
import pytest
import torch

import dispatch_grouped_gemm_gb300 as hmm
from tests import open_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"

# (T, H, E, K): one token; more experts than slots; rows of an odd number of elements
# (one element per access), pieces that end inside a warp's vectors, several hundred
# thousand warps
SHAPES = [(1, 64, 4, 1), (1, 7168, 256, 8), (3, 8, 5, 2), (17, 1000, 30, 8), (33, 77, 8, 3),
          (129, 520, 64, 32), (2050, 2048, 16, 6), (5000, 24, 1024, 4)]
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def problem(T, H, E, K, dtype, seed=0, bad=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    ids = torch.rand((T, E), generator=g, device=DEV).argsort(1)[:, :K].int()
    if bad:
        out = torch.rand((T, K), generator=g, device=DEV) < bad
        ids = torch.where(out, torch.where(ids % 2 == 0, E + 3, -1).int(), ids)
    x = torch.randn((T, H), generator=g, device=DEV).to(dtype)
    return ids.contiguous(), x, g


def clear_status():
    return hmm.hmm_status(hmm.Context.for_device(torch.device(DEV, 0)).handle)


@pytest.mark.parametrize("shape", SHAPES)
def test_route(shape):
    T, H, E, K = shape
    ids, _, _ = problem(T, 8, E, K, torch.float32)
    r = hmm.moe_route(ids, E)
    offsets, slot2row, row2slot = ref.route(ids, E)
    assert torch.equal(r.offsets.long(), offsets)
    assert torch.equal(r.counts.long(), offsets[1:] - offsets[:-1])
    assert torch.equal(r.slot2row.long(), slot2row)
    assert torch.equal(r.row2slot.long(), row2slot)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_dispatch(shape, dtype):
    T, H, E, K = shape
    ids, x, g = problem(*shape, dtype)
    r = hmm.moe_route(ids, E)
    x.requires_grad_()
    rows = hmm.moe_dispatch(x, r)
    assert rows.dtype == dtype
    assert torch.equal(rows.detach().double(), ref.dispatch(x.detach(), r.slot2row.long()))
    d_rows = torch.randn(rows.shape, generator=g, device=DEV).to(dtype)
    (dx,) = torch.autograd.grad(rows, x, d_rows)
    # K fp32 additions, each off by at most 2^-24 of a partial sum
    slack = ref.dispatch_grad(d_rows.abs(), r.slot2row.long()) * K * 2.0 ** -24
    ref.assert_close("dx", dx, ref.dispatch_grad(d_rows, r.slot2row.long()), slack)


@pytest.mark.parametrize("wdtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_combine(shape, dtype, wdtype):
    T, H, E, K = shape
    ids, dy, g = problem(*shape, dtype)
    r = hmm.moe_route(ids, E)
    at = r.slot2row.long()
    rows = torch.randn((T * K, H), generator=g, device=DEV).to(dtype).requires_grad_()
    w = torch.randn((T, K), generator=g, device=DEV).to(wdtype).requires_grad_()
    y = hmm.moe_combine(rows, r, w)
    rd, wd = rows.detach(), w.detach()
    slack = ref.combine(rd.abs(), at, wd.abs()) * K * 2.0 ** -24
    ref.assert_close("y", y.detach(), ref.combine(rd, at, wd), slack)
    d_rows, dw = torch.autograd.grad(y, (rows, w), dy)
    want_rows, want_w = ref.combine_grad(rd, at, wd, dy)
    ref.assert_close("d_rows", d_rows, want_rows, want_rows.abs() * 2.0 ** -24)
    _, weight = ref.combine_grad(rd.abs(), at, wd, dy.abs())
    ref.assert_close("d_w", dw, want_w, weight * H * 2.0 ** -24)


@pytest.mark.parametrize("shape", [(17, 1000, 30, 8), (33, 77, 8, 3), (2050, 128, 16, 6)])
def test_invalid_ids(shape):
    """Slots of invalid ids have no row, add nothing and get no gradient; the rows
    behind the last expert's are zeros."""
    T, H, E, K = shape
    clear_status()
    ids, x, g = problem(*shape, torch.bfloat16, bad=0.2)
    ids[1] = -5  # a token with no expert at all
    r = hmm.moe_route(ids, E)
    assert clear_status() == (hmm.HMM_ERR_EXPERT_ID, hmm.HMM_STATUS_EXPERT_ID)
    offsets, slot2row, row2slot = ref.route(ids, E)
    assert torch.equal(r.offsets.long(), offsets) and torch.equal(r.slot2row.long(), slot2row)
    assert torch.equal(r.row2slot[:row2slot.numel()].long(), row2slot)
    torch.full((T * K, H), float("nan"), dtype=torch.bfloat16, device=DEV)  # stale memory
    x.requires_grad_()
    rows = hmm.moe_dispatch(x, r)
    assert torch.equal(rows.detach().double(), ref.dispatch(x.detach(), slot2row))
    # what lies behind the last expert's rows is not read
    filled = rows.detach().clone()
    filled[int(offsets[E]):] = float("nan")
    w = torch.randn((T, K), generator=g, device=DEV)
    filled.requires_grad_()
    w.requires_grad_()
    y = hmm.moe_combine(filled, r, w)
    assert bool(torch.isfinite(y).all()) and not bool(y[1].any())
    dy = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
    d_rows, dw = torch.autograd.grad(y, (filled, w), dy)
    assert not bool(d_rows[int(offsets[E]):].any()) and not bool(dw[slot2row < 0].any())
    want_rows, _ = ref.combine_grad(rows.detach(), slot2row, w.detach(), dy)
    ref.assert_close("d_rows", d_rows, want_rows, want_rows.abs() * 2.0 ** -24)
    (dx,) = torch.autograd.grad(rows, x, filled.detach())
    assert bool(torch.isfinite(dx).all()) and not bool(dx[1].any())


def test_empty_batch():
    r = hmm.moe_route(torch.empty((0, 4), dtype=torch.int32, device=DEV), 8)
    assert r.offsets.tolist() == [0] * 9 and r.counts.tolist() == [0] * 8
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV, requires_grad=True)
    rows = hmm.moe_dispatch(x, r)
    assert rows.shape == (0, 64)
    w = torch.empty((0, 4), device=DEV, requires_grad=True)
    y = hmm.moe_combine(rows, r, w)
    assert y.shape == (0, 64)
    dx, dw = torch.autograd.grad(y.sum(), (x, w))
    assert dx.shape == x.shape and dw.shape == w.shape


def test_strides():
    """Rows of x and dy that lie apart, that are broadcast, that start off 16 bytes,
    and columns that are no unit stride."""
    T, H, E, K = 37, 128, 8, 3
    ids, _, g = problem(T, H, E, K, torch.bfloat16)
    r = hmm.moe_route(ids, E)
    wide = torch.randn((T, 3 * H + 5), generator=g, device=DEV).to(torch.bfloat16)
    rows = torch.randn((T * K, H), generator=g, device=DEV).to(torch.bfloat16).requires_grad_()
    w = torch.rand((T, K), generator=g, device=DEV).requires_grad_()
    y = hmm.moe_combine(rows, r, w)
    for x in (wide[:, :H], wide[:, 1:H + 1], wide[:, ::3][:, :H], wide[0, :H].expand(T, H)):
        dense = x.clone(memory_format=torch.contiguous_format)
        assert torch.equal(hmm.moe_dispatch(x, r), hmm.moe_dispatch(dense, r))
        a_rows, a_w = torch.autograd.grad(y, (rows, w), x, retain_graph=True)
        b_rows, b_w = torch.autograd.grad(y, (rows, w), dense, retain_graph=True)
        assert torch.equal(a_rows, b_rows)
        # (another number of elements per access sums d_w in another order)
        _, mass = ref.combine_grad(rows.detach().abs(), r.slot2row.long(), w.detach(), dense.abs())
        assert bool(((a_w - b_w).abs() <= mass * 2 * H * 2.0 ** -24).all())
    apart = torch.randn((T * K, 2 * H), generator=g, device=DEV).to(torch.bfloat16)[:, :H]
    assert torch.equal(hmm.moe_combine(apart, r, w.detach()),
                       hmm.moe_combine(apart.contiguous(), r, w.detach()))
    wt = w.detach().T.contiguous().T
    assert torch.equal(hmm.moe_combine(rows.detach(), r, wt), y.detach())


def test_special_values():
    """Infinities and NaN stay in the tokens that have them."""
    T, H, E, K = 9, 64, 4, 2
    ids, x, g = problem(T, H, E, K, torch.float32)
    r = hmm.moe_route(ids, E)
    x[3, 5], x[4, 6] = float("inf"), float("nan")
    rows = hmm.moe_dispatch(x, r)
    y = hmm.moe_combine(rows, r, torch.ones((T, K), device=DEV))
    bad = ~torch.isfinite(y)
    assert bool(bad[3, 5]) and bool(torch.isnan(y[4, 6])) and int(bad.sum()) == 2


def test_second_derivative_is_refused():
    ids, x, g = problem(5, 16, 4, 2, torch.float32)
    r = hmm.moe_route(ids, 4)
    x.requires_grad_()
    rows = hmm.moe_dispatch(x, r)
    (dx,) = torch.autograd.grad(rows.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="no second derivative"):
        dx.sum().backward()
    w = torch.ones((5, 2), device=DEV, requires_grad=True)
    y = hmm.moe_combine(rows.detach(), r, w)
    (dw,) = torch.autograd.grad(y.square().sum(), w, create_graph=True)
    with pytest.raises(RuntimeError, match="no second derivative"):
        dw.sum().backward()


def test_gradients_against_differences():
    """Both maps are linear in rows and weights: a difference is exact up to fp32."""
    T, H, E, K = 6, 40, 4, 3
    ids, x, g = problem(T, H, E, K, torch.float32)
    r = hmm.moe_route(ids, E)
    w = torch.rand((T, K), generator=g, device=DEV)
    x.requires_grad_()
    w.requires_grad_()
    dy = torch.randn((T, H), generator=g, device=DEV)

    def f(x, w):
        return (hmm.moe_combine(hmm.moe_dispatch(x, r), r, w).double() * dy).sum()

    dx, dw = torch.autograd.grad(f(x, w), (x, w))
    px, pw = torch.randn_like(x), torch.randn_like(w)
    with torch.no_grad():
        nx = (f(x + px, w) - f(x - px, w)) / 2
        nw = (f(x, w + pw) - f(x, w - pw)) / 2
    # sums of T * H * K products of order 1 in fp32
    tol = T * H * K * 2.0 ** -20
    assert abs(nx.item() - (dx.double() * px).sum().item()) < tol
    assert abs(nw.item() - (dw.double() * pw).sum().item()) < tol
