"""The float64 forms in oracle/layer.py: their gradients against central
differences of their forward passes, and hand-checked corner cases."""
import numpy as np
import pytest

from oracle import layer


def _rng(k):
    return np.random.default_rng([77, k])


def _difference(f, at, direction, h=1e-5):
    """Central difference of the scalar f along `direction`; its error is
    about h^2 |f'''| / 6 + 2^-52 |f| / h, under 1e-7 of these O(10) values."""
    return (f(at + h * direction) - f(at - h * direction)) / (2 * h)


def test_grouped_gradients_against_differences():
    g = _rng(0)
    off = [1, 4, 4, 9]                     # rows 0 and 9 belong to no run, run 1 is empty
    x, w, dy = g.standard_normal((10, 5)), g.standard_normal((3, 4, 5)), g.standard_normal((10, 4))

    def loss(x, w):
        return (dy * layer.grouped(x, w, off)[0]).sum()

    vx, vw = g.standard_normal(x.shape), g.standard_normal(w.shape)
    dx, dw = layer.grouped_dgrad(dy, w, off)[0], layer.grouped_wgrad(dy, x, off)[0]
    assert abs(_difference(lambda a: loss(a, w), x, vx) - (dx * vx).sum()) < 1e-7
    assert abs(_difference(lambda a: loss(x, a), w, vw) - (dw * vw).sum()) < 1e-7
    assert not dx[0].any() and not dx[9].any() and not dw[1].any()


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
def test_activation_slopes_against_differences(act):
    z = np.concatenate([_rng(1).standard_normal(64) * 3, [-40.0, 40.0, 0.5, -0.5]])
    d = (layer.activation(act, z + 1e-5) - layer.activation(act, z - 1e-5)) / 2e-5
    assert np.abs(d - layer.slope(act, z)).max() < 1e-7
    assert layer.slope("relu", np.zeros(1))[0] == 0


def test_layer_norm_gradients_against_differences():
    g = _rng(2)
    x, w, b, dy = (g.standard_normal(s) for s in ((6, 11), 11, 11, (6, 11)))

    def loss(x, w, b):
        return (dy * layer.layer_norm(x, w, b, 1e-5)[0]).sum()

    _, mean, rstd = layer.layer_norm(x, w, b, 1e-5)
    dx, dw, db = layer.layer_norm_backward(dy, x, w, mean, rstd)
    vx, vw, vb = g.standard_normal(x.shape), g.standard_normal(11), g.standard_normal(11)
    assert abs(_difference(lambda a: loss(a, w, b), x, vx) - (dx * vx).sum()) < 1e-7
    assert abs(_difference(lambda a: loss(x, a, b), w, vw) - dw @ vw) < 1e-7
    assert abs(_difference(lambda a: loss(x, w, a), b, vb) - db @ vb) < 1e-7


def test_layer_norm_of_equal_values():
    y, mean, rstd = layer.layer_norm(np.full((1, 4), 3.0), np.ones(4), np.arange(4.0), 0.25)
    assert mean[0] == 3 and rstd[0] == 2 and np.array_equal(y[0], np.arange(4.0))


def test_combine_gradients_against_differences():
    g = _rng(3)
    rows = np.array([[0, 3], [-1, 5], [2, -1], [-1, -1]])
    y, p, dout = g.standard_normal((6, 7)), g.standard_normal((4, 2)), g.standard_normal((4, 7))

    def loss(y, p):
        return (dout * layer.combine(y, rows, p)).sum()

    dy, dp = layer.combine_backward(dout, y, rows, p)
    vy, vp = g.standard_normal(y.shape), g.standard_normal(p.shape)
    assert abs(_difference(lambda a: loss(a, p), y, vy) - (dy * vy).sum()) < 1e-7
    assert abs(_difference(lambda a: loss(y, a), p, vp) - (dp * vp).sum()) < 1e-7
    assert not dp[3].any() and not dy[1].any() and not layer.combine(y, rows, p)[3].any()
