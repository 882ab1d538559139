"""The oracle's activations where they are small, against their asymptotic forms."""
import numpy as np

from oracle import products as op


def test_gelu():
    a = np.array([8.0, 12.5, 20.0, 35.0])
    phi = np.exp(-a * a / 2) / np.sqrt(2 * np.pi)
    y, d = op.act("gelu", -a)
    low, high = 1 - a ** -2, 1 - a ** -2 + 3 * a ** -4  # of a Phi(-a) / phi(a)
    assert (-y / phi >= low * (1 - 1e-12)).all() and (-y / phi <= high * (1 + 1e-12)).all()
    # Phi(-a) - a phi(a)
    assert (-d / phi >= a - high / a * (1 + 1e-12)).all() and (-d / phi <= a - low / a * (1 - 1e-12)).all()


def test_sigmoids():
    for name, z, inner in (("silu", lambda g: g, lambda g: 1),
                           ("gelu_tanh", lambda g: np.sqrt(8 / np.pi) * (g + 0.044715 * g ** 3),
                            lambda g: np.sqrt(8 / np.pi) * (1 + 3 * 0.044715 * g * g))):
        g = np.array([-8.0, -9.5, -11.0]) * (5 if name == "silu" else 1)
        s = np.exp(z(g))
        y, d = op.act(name, g)
        assert np.abs(y / (g * s) - 1).max() < 2 * s.max() + 1e-13
        assert np.abs(d / (s * (1 + g * inner(g))) - 1).max() < 4 * s.max() + 1e-13


def test_large_gates_are_finite():
    g = np.array([200.0, 1e4, 1e19, 3e38])
    with np.errstate(all="raise", under="ignore"):
        for name in ("silu", "gelu", "gelu_tanh"):
            y, d = op.act(name, g)
            assert (y == g).all() and (d == 1).all()
            y, d = op.act(name, -g)
            assert np.abs(y).max() < 1e-80 and np.abs(d).max() < 1e-80
