"""What pins the fp64 oracle of the norm: rows of known mean square, and
differences for its gradient."""
import numpy as np

from oracle import norm as onorm


def test_rows_have_unit_mean_square():
    h = np.random.default_rng(0).standard_normal((5, 40)) * 7.0
    y = onorm.forward(h, np.ones(40), 0.0)
    np.testing.assert_allclose((y * y).mean(1), 1.0, rtol=1e-12)
    np.testing.assert_allclose(onorm.forward(3.0 * h, np.ones(40), 0.0), y, rtol=1e-12)
    np.testing.assert_allclose(onorm.forward(np.zeros((1, 8)), np.ones(8), 1e-6), 0.0)
    # mean square 12.5 + eps 12.5: rms 5
    y = onorm.forward(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), 12.5)
    np.testing.assert_allclose(y, [[0.6, 1.6]], rtol=1e-15)


def test_scales():
    y = np.array([[1.0, -448.0, 2.0, 0.0, 0.0]])
    assert onorm.scales(y, 0).tolist() == [[1.0]]
    assert onorm.scales(y, 3).tolist() == [[1.0, 2.0 ** -100 / 448.0]]


def test_gradient_against_differences():
    r = np.random.default_rng(1)
    h, w, dy, dho = (r.standard_normal(s) for s in ((3, 7), 7, (3, 7), (3, 7)))

    def loss(h, w):
        return float((onorm.forward(h, w, 0.1) * dy).sum() + (h * dho).sum())
    dh, dw, _, _ = onorm.backward(dy, h, w, 0.1, dho)
    e = 1e-6
    for got, at in ((dh, 0), (dw, 1)):
        for i in np.ndindex(got.shape):
            a, b = [h.copy(), w.copy()], [h.copy(), w.copy()]
            a[at][i] += e
            b[at][i] -= e
            assert abs((loss(*a) - loss(*b)) / (2 * e) - got[i]) < 1e-7
