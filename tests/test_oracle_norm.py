"""The norm oracle: its gradient against central differences, and the closed
forms of rows that have one."""
import numpy as np
import pytest

from oracle import norm as N


@pytest.mark.parametrize("T,d,eps", [(1, 8, 1e-6), (3, 16, 1e-2), (4, 7, 0.5)])
def test_gradient_is_the_difference_quotient(T, d, eps):
    rng = np.random.default_rng(T * 100 + d)
    x, resid, w = rng.normal(size=(T, d)), rng.normal(size=(T, d)), 1 + 0.3 * rng.normal(size=d)
    du, dr = rng.normal(size=(T, d)), rng.normal(size=(T, d))

    def loss(x, w):
        r, _, u = N.rmsnorm(x, resid, w, eps)
        return np.sum(du * u) + np.sum(dr * r)

    r, c, _ = N.rmsnorm(x, resid, w, eps)
    dx, dw = N.rmsnorm_backward(du, r, w, c, dr)
    # the quotient's own error: h^2 / 6 times a third derivative of a few tens, and 1e-16 / h
    h = 1e-5
    for (t, j) in [(0, 0), (T - 1, d - 1), (T // 2, d // 2)]:
        e = np.zeros_like(x)
        e[t, j] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[t, j]) < 1e-7
    for j in range(d):
        e = np.zeros_like(w)
        e[j] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[j]) < 1e-7


def test_constant_rows():
    w = np.array([1.0, 2.0, -3.0, 0.5])
    _, c, u = N.rmsnorm(np.full((2, 4), 5.0), None, w, 0.0)
    np.testing.assert_allclose(c, 0.2)
    np.testing.assert_allclose(u, np.stack([w, w]))
    _, _, u = N.rmsnorm(np.zeros((1, 4)), None, w, 1e-6)
    assert not u.any()
    # without eps the norm does not see the row's scale, so its gradient has no part along the row
    r, c, _ = N.rmsnorm(np.arange(1.0, 5.0)[None], None, w, 0.0)
    dx, _ = N.rmsnorm_backward(np.ones((1, 4)), r, w, c)
    assert abs(np.sum(dx * r)) < 1e-12
