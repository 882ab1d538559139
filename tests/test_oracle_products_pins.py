"""The products' oracle against what the definitions fix."""
import numpy as np
import pytest

from oracle import products as op


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh", "identity"])
def test_slopes_are_differences(name):
    g = np.linspace(-6, 6, 241)
    h = 1e-5
    d = (op.act(name, g + h)[0] - op.act(name, g - h)[0]) / (2 * h)
    assert np.abs(d - op.act(name, g)[1]).max() < 1e-9
    assert np.abs(op.act(name, np.array([0.0, 40.0]))[0] - [0.0, 40.0]).max() < 1e-12  # act(0) = 0, act(g) -> g


def test_gelu_forms_are_near():
    g = np.linspace(-6, 6, 241)
    assert np.abs(op.act("gelu", g)[0] - op.act("gelu_tanh", g)[0]).max() < 5e-4


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh", "identity"])
def test_gradient_is_differences(name):
    r = np.random.default_rng(0)
    M, D, F = 3, 5, 4
    p = [r.standard_normal(s) for s in ((M, D), (F, D), (F, D))]
    dy = r.standard_normal((M, F))
    _, g, u, _, _ = op.gated(*p, name)
    grads = op.gated_backward(dy, *p, g, u, name)[:3]
    for i, want in enumerate(grads):
        d = r.standard_normal(p[i].shape)
        h = 1e-6
        up, down = [list(p) for _ in range(2)]
        up[i], down[i] = p[i] + h * d, p[i] - h * d
        slope = ((op.gated(*up, name)[0] - op.gated(*down, name)[0]) * dy).sum() / (2 * h)
        assert abs(slope - (want * d).sum()) < 1e-7


def test_scales_by_hand():
    x = np.zeros((130, 256))
    x[0, 0], x[129, 127], x[5, 200] = -896.0, 448.0, 0.5
    assert op.scales(x, 128).shape == (2, 2)
    assert (op.scales(x, 128) == [[2.0, 0.5 / 448], [1.0, 2.0 ** -100 / 448]]).all()
    assert op.scales(x, 1)[0, 0] == 2.0 and op.scales(x, 1)[5, 1] == 0.5 / 448
    assert (op.values(np.ones((130, 256)), op.scales(x, 128), 128)[:, ::128][[0, 128]] == op.scales(x, 128)).all()
