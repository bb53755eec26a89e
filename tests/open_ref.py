"""The open expert layer and the orthogonalised update in plain 64-bit torch, and how
far a result that is rounded once may be from them."""
import torch

QUINTIC = (3.4445, -4.7750, 2.0315)


def route(ids, E):
    """(offsets, slot2row [T, K], row2slot) of ids [T, K], stable."""
    T, K = ids.shape
    flat = ids.flatten().long()
    ok = (flat >= 0) & (flat < E)
    row2slot = torch.nonzero(ok).flatten()
    row2slot = row2slot[torch.argsort(flat[row2slot], stable=True)]
    slot2row = torch.full((T * K,), -1, dtype=torch.long, device=ids.device)
    slot2row[row2slot] = torch.arange(row2slot.numel(), device=ids.device)
    counts = torch.bincount(flat[ok], minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.long, device=ids.device)
    offsets[1:] = counts.cumsum(0)
    return offsets, slot2row.view(T, K), row2slot


def dispatch(x, slot2row):
    T, K = slot2row.shape
    rows = torch.zeros((T * K, x.shape[1]), dtype=torch.float64, device=x.device)
    for k in range(K):
        ok = slot2row[:, k] >= 0
        rows[slot2row[ok, k]] = x[ok].double()
    return rows


def dispatch_grad(d_rows, slot2row):
    picked = d_rows.double()[slot2row.clamp(min=0)]
    return torch.where((slot2row >= 0).unsqueeze(2), picked, 0.0).sum(1)


def combine(rows, slot2row, w):
    picked = torch.where((slot2row >= 0).unsqueeze(2), rows.double()[slot2row.clamp(min=0)], 0.0)
    return (picked * w.double().unsqueeze(2)).sum(1)


def combine_grad(rows, slot2row, w, dy):
    ok = slot2row >= 0
    picked = torch.where(ok.unsqueeze(2), rows.double()[slot2row.clamp(min=0)], 0.0)
    dw = (picked * dy.double().unsqueeze(1)).sum(2)
    d_rows = torch.zeros(rows.shape, dtype=torch.float64, device=rows.device)
    for k in range(slot2row.shape[1]):
        i = ok[:, k]
        d_rows[slot2row[i, k]] = w[i, k].double().unsqueeze(1) * dy[i].double()
    return d_rows, dw


def grouped_mm(x, w, offsets):
    o = [int(v) for v in offsets]
    y = torch.zeros((x.shape[0], w.shape[2]), dtype=torch.float64, device=x.device)
    for e in range(w.shape[0]):
        y[o[e]:o[e + 1]] = x[o[e]:o[e + 1]].double() @ w[e].double()
    return y


def grouped_mm_dw(x, dy, offsets):
    o = [int(v) for v in offsets]
    return torch.stack([x[o[e]:o[e + 1]].double().T @ dy[o[e]:o[e + 1]].double()
                        for e in range(len(o) - 1)])


def orthogonalize(g, steps=5, coefficients=QUINTIC, eps=1e-7, scale=1.0, rounded=False):
    """In 64 bits; with `rounded`, the operands of the products rounded to 11 bits
    and X between the steps to 22, as the kernels hold them (their range aside)."""
    if not isinstance(coefficients[0], (tuple, list)):
        coefficients = [coefficients] * steps

    def bits(v, n):
        m, e = torch.frexp(v)
        return torch.ldexp(torch.round(torch.ldexp(m, torch.tensor(n))), e - n)

    out = []
    for x in g.double().reshape(-1, *g.shape[-2:]):
        tall = x.shape[0] > x.shape[1]
        x = x.T if tall else x
        x = x / (x.norm() + eps)
        one = torch.eye(x.shape[0], dtype=torch.float64, device=x.device)
        for a, b, c in coefficients:
            if rounded:
                hi = bits(x, 11)
                s = bits(hi @ hi.T, 11)
                p = bits(b * s + c * (s @ s) + a * one, 11)
                x = bits(p @ hi + a * (x - hi), 22)
            else:
                s = x @ x.T
                x = a * x + (b * s + c * (s @ s)) @ x
        out.append((x.T if tall else x) * scale)
    return torch.stack(out).view(g.shape)


def half_step(ref, dtype):
    """One rounding to dtype: half a step relative to the value, half the smallest
    step below the normal range."""
    f = torch.finfo(dtype)
    return ref.abs() * (f.eps / 2) + f.tiny * f.eps / 2


def assert_close(name, got, ref, slack, dtype=None):
    """|got - ref| <= one rounding to the result's type of a value that is off by at
    most `slack`."""
    dtype = dtype or got.dtype
    got = got.double()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    err = (got - ref).abs()
    lim = half_step(ref.abs() + slack, dtype) + slack
    bad = ~(err <= lim)
    if bool(bad.any()):
        i = int(torch.argmax(torch.where(torch.isfinite(err), err / lim, torch.inf)))
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} outside; at {i}: got "
                             f"{got.flatten()[i].item()!r}, want {ref.flatten()[i].item()!r}, "
                             f"limit {lim.flatten()[i].item():.3g}")
