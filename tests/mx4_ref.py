"""Microscaled 4-bit blocks and the experts' products with them, in 64 bits
(numpy), straight from the definition."""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def blocks(v):
    """[..., K] to [..., K/32, 32], zero-padded."""
    v = np.asarray(v, np.float64)
    pad = -v.shape[-1] % 32
    v = np.concatenate([v, np.zeros(v.shape[:-1] + (pad,))], -1)
    return v.reshape(v.shape[:-1] + (-1, 32))


def scale_bytes(v):
    b = np.abs(blocks(v))
    finite = np.isfinite(b).all(-1)
    amax = np.where(finite, np.where(np.isfinite(b), b, 0).max(-1), 1.0)
    _, e = np.frexp(amax)  # amax = m 2^e, m in [.5, 1)
    s = np.where(amax > 0, np.clip(e - 3, -127, 127), -127) + 127
    return np.where(finite, s, 255).astype(np.uint8)


def scale_values(s):
    return np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127))


def nearest(m):
    """Indices into GRID of magnitudes m >= 0: nearest, ties to the even code."""
    lo = np.clip(np.searchsorted(GRID, m, side="right") - 1, 0, 7)
    hi = np.minimum(lo + 1, 7)
    dl, dh = m - GRID[lo], GRID[hi] - m
    up = (dh < dl) | ((dh == dl) & (lo % 2 == 1))
    return np.where(up, hi, lo)


def quantize(v):
    """(codes [..., Kp], scale bytes [..., Kp/32]); codes of NaN blocks are not defined."""
    b = blocks(v)
    s = scale_bytes(v)
    inv = np.where(s == 255, 0.0, 1.0 / scale_values(np.where(s == 255, 127, s)))
    m = np.where(np.isfinite(b), b, 0) * inv[..., None]
    c = nearest(np.abs(m)) + 8 * np.signbit(m)
    return c.reshape(c.shape[:-2] + (-1,)).astype(np.uint8), s


def values(codes, s):
    v = np.where(codes >= 8, -1.0, 1.0) * GRID[codes & 7]
    v = v.reshape(v.shape[:-1] + (-1, 32)) * scale_values(s)[..., None]
    return v.reshape(v.shape[:-2] + (-1,))


def rounded(v):
    """v [..., K] rounded to 4-bit blocks along its last axis."""
    k = np.asarray(v).shape[-1]
    return values(*quantize(v))[..., :k]


def store(codes, s):
    """codes [N, Kp] and scales [N, Kp/32] in their storage."""
    n, kp = codes.shape
    packed = codes[:, 0::2] | (codes[:, 1::2] << 4)
    nt, kt = -(-n // 128), -(-kp // 128)
    t = np.zeros((nt, kt, 512), np.uint8)
    for r in range(n):
        for c in range(kp // 32):
            t[r // 128, c // 4, r % 32 * 16 + r // 32 % 4 * 4 + c % 4] = s[r, c]
    return packed, t


def gate_up_rows(w):
    """[K, 2I] columns to stored rows [2 Ip, K]: 32 gate rows, 32 up rows in turn."""
    k, n = w.shape
    i = n // 2
    ip = -(-i // 32) * 32
    g = np.zeros((2, ip, k))
    g[0, :i], g[1, :i] = w[:, :i].T, w[:, i:].T
    return g.reshape(2, ip // 32, 32, k).transpose(1, 0, 2, 3).reshape(2 * ip, k)


def ffn(x, ids, w, W1, W2):
    """y [T, H] from x [T, H], ids and w [T, K] and the 4-bit values of the
    experts W1 [E, H, 2I], W2 [E, I, H]."""
    x = rounded(x)
    y = np.zeros_like(x)
    I = W2.shape[1]
    for t in range(x.shape[0]):
        for k in range(ids.shape[1]):
            h = x[t] @ W1[ids[t, k]]
            g, u = h[:I], h[I:]
            a = rounded(g / (1 + np.exp(-g)) * u)
            y[t] += w[t, k] * (a @ W2[ids[t, k]])
    return y


def _with_scale(b, s):
    """Blocks b [..., 32] rounded with the scale bytes s."""
    sv = scale_values(s)[..., None]
    return np.sign(b) * GRID[nearest(np.abs(b) / sv)] * sv


def rounded_range(v, dv):
    """(rounded(v), the largest change of it when v moves by up to dv): what a
    value beside a rounding boundary, or a block maximum beside a power of two,
    may become when v is computed in fewer bits."""
    b, d = blocks(v), blocks(dv)
    base = _with_scale(b, scale_bytes(v))
    amax = np.abs(b)
    lo_v = np.maximum(amax - d, 0).max(-1, keepdims=True)
    hi_v = (amax + d).max(-1, keepdims=True)
    out = np.zeros_like(base)
    for top in (lo_v, hi_v):
        s = scale_bytes(np.broadcast_to(top, b.shape).reshape(v.shape[:-1] + (-1,)))
        for sign in (-1, 0, 1):
            out = np.maximum(out, np.abs(_with_scale(b + sign * d, s) - base))
    k = v.shape[-1]
    flat = v.shape[:-1] + (-1,)
    return base.reshape(flat)[..., :k], out.reshape(flat)[..., :k]


def ffn_bounded(x, ids, w, W1, W2):
    """(y, an elementwise bound of what fp32 products, their sums in fp32 and
    bf16 rows of expert outputs may add)."""
    x = rounded(x)
    y, lim = np.zeros_like(x), np.zeros_like(x)
    I = W2.shape[1]
    eps = 2.0 ** -20  # fp32 products and sums of up to a few thousand terms
    for t in range(x.shape[0]):
        for k in range(ids.shape[1]):
            if not 0 <= ids[t, k] < W1.shape[0]:
                continue
            h = x[t] @ W1[ids[t, k]]
            e = eps * (np.abs(x[t]) @ np.abs(W1[ids[t, k]]))
            g, u, eg, eu = h[:I], h[I:], e[:I], e[I:]
            sg = 1 / (1 + np.exp(-g))
            v = g * sg * u
            # |silu'| <= 1.1; the exponential and the division: 1e-6 relative,
            # and 2^-24 |g| from the exponent's own rounding
            dv = 1.1 * eg * np.abs(u) + np.abs(g * sg) * eu + (2e-6 + 2e-7 * np.abs(g)) * np.abs(v)
            a, da = rounded_range(v[None], dv[None])
            o = a[0] @ W2[ids[t, k]]
            mag = np.abs(a[0]) @ np.abs(W2[ids[t, k]])
            y[t] += w[t, k] * o
            lim[t] += abs(w[t, k]) * (da[0] @ np.abs(W2[ids[t, k]]) + eps * mag
                                      + 2.0 ** -8 * np.abs(o))
    return y, lim + 2.0 ** -8 * np.abs(y) + 1e-30
