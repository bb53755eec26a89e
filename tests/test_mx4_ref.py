"""The 64-bit reference of the 4-bit blocks against what the format fixes."""
import numpy as np

from tests import mx4_ref as ref


def test_rounding_by_brute_force():
    m = np.arange(0, 8.0001, 1 / 64)
    for v, got in zip(m, ref.GRID[ref.nearest(m)]):
        d = np.abs(ref.GRID - v)
        near = [i for i in range(8) if d[i] == d.min()]
        want = near[0] if len(near) == 1 else [i for i in near if i % 2 == 0][0]
        assert got == ref.GRID[want]


def test_scales():
    v = np.zeros((1, 32 * 7))
    v[0, 32], v[0, 64], v[0, 96] = 1.0, 7.99, -8.0
    v[0, 128], v[0, 160], v[0, 192] = np.inf, np.nan, 2.0 ** -140
    assert ref.scale_bytes(v)[0].tolist() == [0, 125, 127, 128, 255, 255, 0]


def test_values_are_fixed_points():
    rng = np.random.default_rng(0)
    v = rng.normal(size=(4, 96)) * np.exp2(rng.integers(-30, 30, size=(4, 1)))
    r = ref.rounded(v)
    assert np.array_equal(ref.rounded(r), r)
    # half a step of the largest interval (4 .. 6), or saturation (up to 8), at most
    s = np.repeat(ref.scale_values(ref.scale_bytes(v)), 32, -1)
    assert (np.abs(v - r) <= 2 * s).all()


def test_gate_up_rows():
    w = np.arange(2.0 * 80).reshape(2, 80)
    r = ref.gate_up_rows(w)
    assert r.shape == (128, 2)
    assert np.array_equal(r[:32], w[:, :32].T) and np.array_equal(r[32:64], w[:, 40:72].T)
    assert np.array_equal(r[64:72], w[:, 32:40].T) and not r[72:96].any()
    assert np.array_equal(r[96:104], w[:, 72:].T) and not r[104:].any()
