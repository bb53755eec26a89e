"""The 64-bit router reference of the GPU tests against what it must satisfy:
its gradient against central differences, closed forms, and rows with closed
experts."""
import numpy as np
import pytest

from tests import gate_ref as ref


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("with_scores", [False, True])
def test_gradient_against_differences(score, renorm, with_scores):
    rng = np.random.default_rng(3)
    T, E, K, scale, h = 4, 9, 3, 1.7, 1e-5
    l = rng.normal(size=(T, E))
    dw = rng.normal(size=(T, K))
    ds = rng.normal(size=(T, E)) if with_scores else None
    ids = ref.select(l, K, np.ones((T, E), bool))

    def loss(v):
        p = ref.scores(v, score)
        out = (ref.weights(p, ids, renorm, scale) * dw).sum()
        return out + ((p * ds).sum() if with_scores else 0.0)

    g, _ = ref.d_logits(l, ids, dw, ds, score, renorm, scale)
    for t in range(T):
        for e in range(E):
            v = l.copy()
            v[t, e] += h
            hi = loss(v)
            v[t, e] -= 2 * h
            # central differences: truncation ~ h^2, rounding ~ 1e-16 / h
            assert abs((hi - loss(v)) / (2 * h) - g[t, e]) < 1e-8


def test_closed_forms():
    l = np.zeros((1, 4))
    assert np.allclose(ref.scores(l, "softmax"), 0.25)
    assert np.allclose(ref.scores(l, "sigmoid"), 0.5)
    ids = ref.select(l, 2, np.ones((1, 4), bool))
    assert ids.tolist() == [[0, 1]]
    assert np.allclose(ref.weights(ref.scores(l, "softmax"), ids, True, 2.0), 1.0)


def test_rows_with_closed_experts():
    l = np.array([[-np.inf, 1.0, -np.inf], [-np.inf] * 3])
    p = ref.scores(l, "softmax")
    assert p[0].tolist() == [0.0, 1.0, 0.0] and not p[1].any()
    ids = ref.select(l, 2, np.ones((2, 3), bool))
    assert ids.tolist() == [[1, 0], [0, 1]]
    assert not ref.weights(p, ids, True, 1.0)[1].any()


def test_groups():
    key = np.array([[5.0, 0.0, 3.0, 3.0, 4.0, 1.0]])
    assert ref.open_experts(key, 3, 1, 1).tolist() == [[True, True, False, False, False, False]]
    assert ref.open_experts(key, 3, 1, 2).tolist() == [[False, False, True, True, False, False]]
