"""fp64 oracle of the 8-bit products, their quantiser and the gated feed-forward
block: plain numpy, from the definitions.  Test infrastructure only."""
from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100
GROUP = 128
_erfc = np.vectorize(math.erfc, otypes=[float])


def scales(x, block):
    """max |x| / 448 per `block` rows x 128 columns."""
    rows = [np.abs(x[i:i + block]) for i in range(0, x.shape[0], block)]
    s = [[r[:, j:j + GROUP].max(1) if block == 1 else r[:, j:j + GROUP].max() for j in range(0, x.shape[1], GROUP)]
         for r in rows]
    s = np.array(s, dtype=float).reshape(len(rows), -1)
    return np.maximum(s, AMAX_FLOOR) / E4M3_MAX


def spread(s, block, shape):
    """Each value's scale."""
    return np.repeat(np.repeat(s, block, 0)[:shape[0]], GROUP if s.shape[1] > 1 else shape[1], 1)[:, :shape[1]]


def values(q, s, block):
    """The values that codes q stand for."""
    return q * spread(s, block, q.shape)


def _sigmoid(z):
    """(1 / (1 + e^-z), 1 / (1 + e^z)), each to the last digits."""
    e = np.exp(-np.abs(z))
    small, large = e / (1 + e), 1 / (1 + e)
    return np.where(z < 0, small, large), np.where(z < 0, large, small)


def act(name, g):
    """(act(g), act'(g)), to the last digits where they are small too."""
    if name == "identity":
        return g, np.ones_like(g)
    if name == "silu":
        s, rest = _sigmoid(g)
        return g * s, s * (1 + g * rest)
    if name == "gelu":
        c = 0.5 * _erfc(-g / math.sqrt(2))
        return g * c, c + g * np.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    # (1 + tanh z) / 2 = 1 / (1 + e^-2z)
    k = 2 * math.sqrt(2 / math.pi)
    s, rest = _sigmoid(k * (g + 0.044715 * g ** 3))
    return g * s, s + g * s * rest * k * (1 + 3 * 0.044715 * g * g)


def gated(x, wg, wu, name):
    """(y, g, u, sums of the absolute terms of g and of u)."""
    g, u = x @ wg.T, x @ wu.T
    return act(name, g)[0] * u, g, u, np.abs(x) @ np.abs(wg).T, np.abs(x) @ np.abs(wu).T


def gated_backward(dy, x, wg, wu, g, u, name):
    """(dx, dWg, dWu, dg, du)."""
    a, d = act(name, g)
    dg, du = dy * u * d, dy * a
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, dg, du
