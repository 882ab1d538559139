"""The activations' relative accuracy where they are small, and their slopes',
with bounds from the arithmetic.

n = 2^-24, half a step of fp32.  e^z is the hardware's 2^x (4 n off) of z log2(e),
whose roundings move it by n |z| each: the constant's and the product's, gelu's
square's, and of gelu_tanh four in the cubic and three in the constant; R(z) = k n
|z| + 4 n with k = 2 (silu), 3 (gelu), 8 (gelu_tanh).  s = 1 / (1 + e^-z) takes (1 - s)
R of it and 3 n by its sum and quotient (2 n for the hardware's 1 / x); where e^-z < n / 4
it is 1, e^-z off.  Phi(-|g|) is R of its exponential off, 4 n for the fit and 26 n for
its arithmetic.  What falls below 2^-126 is taken for zero.  Each product and sum adds n.
"""
import numpy as np
import pytest

from oracle import products as op

pytestmark = pytest.mark.gpu

N, TINY = 2.0 ** -24, 2.0 ** -126
K = {"silu": 2, "gelu": 3, "gelu_tanh": 8}


def bounds(act, g):
    """(error of act(g), error of act'(g)) in fp32, from fp32 g."""
    y, d = op.act(act, g)
    a = np.abs(g)
    if act == "gelu":
        R = K[act] * N * g * g / 2 + 4 * N
        phi, tail = np.exp(-g * g / 2) / np.sqrt(2 * np.pi), np.where(a > 0, op.act(act, -a)[0] / -np.maximum(a, 1e-300), 0.5)
        c = np.where(g < 0, tail, 1 - tail)
        dc = tail * (R + 30 * N) + N * c + TINY
        # past 20 the exponential is zero and what is left of it is below e^-200
        cut = np.minimum(a, 20) * TINY
        return a * np.where(a < 20, dc, N * c) + N * np.abs(y) + cut, \
            dc + a * phi * (R + 3 * N) + 2 * N * np.abs(d) + cut
    if act == "silu":
        z, inner, cut = a, np.ones_like(g), np.minimum(a, 128) * TINY
    else:
        k = 2 * np.sqrt(2 / np.pi)
        b = np.minimum(a, 1e6)  # cubes past it: s is 1 or 0
        z, inner = k * (b + 0.044715 * b ** 3), k * (1 + 3 * 0.044715 * b * b)
        cut = np.minimum(a, 20) * np.minimum(inner, 100) * TINY
    R = K[act] * N * z + 4 * N
    e = np.exp(-z)
    s, rest = np.where(g < 0, e, 1) / (1 + e), np.where(g < 0, 1, e) / (1 + e)
    ds = np.where((g > 0) & (e < N / 4), e, s * (rest * R + 3 * N)) + 2 * TINY
    dy = np.where(a < 1e3, a * ds, 0) + N * np.abs(y) + cut
    dr = np.where(a < 1e3, ds + N * rest, 0)
    if act == "silu":  # s (1 + g rest)
        size = s * (1 + a * rest)
        return dy, ds * (1 + a * rest) + s * np.where(a < 1e3, a * dr, 0) + 3 * N * size + 2 * cut
    size = np.abs(y) * rest * inner  # y rest inner + s
    return dy, dy * rest * inner + np.where(a < 1e3, np.abs(y) * dr * inner, 0) + 6 * N * size + ds + N * np.abs(d) + 2 * cut


def gates(count, seed):
    """fp32 gates from -100 to 100, more of them near zero and in the tails, and large ones."""
    r = np.random.default_rng(seed)
    g = np.concatenate([[0.0, -0.75, -5.5, -9.0, -12.5, -13.3, -87.0, -104.0, 1e4, -1e4, 5.0, 9.0, 20.0, 88.0],
                        r.uniform(-14, 14, count), r.uniform(-100, 100, count), r.normal(0, 1, count)])
    return np.float32(r.permutation(g)[:count])


@pytest.mark.parametrize("act", list(K))
@pytest.mark.parametrize("M,F", [(20, 16), (300, 16), (600, 2560)])
def test_forward_tails(act, M, F):
    """The scale of a row of equal values of y = act(g) 1 shows |act(g)| in fp32."""
    import torch
    import hyena_long_convolution_b200 as hy
    g = gates(M, M)
    e4m3 = torch.float8_e4m3fn
    x, wg, wu = torch.zeros(M, 256), torch.zeros(F, 256), torch.zeros(F, 256)
    x[:, 0] = x[:, 128] = wg[:, 0] = wu[:, 128] = 1.0
    sx = torch.ones(M, 2)
    sx[:, 0] = torch.from_numpy(g)
    one = torch.ones(-(-F // 128), 2, device="cuda")
    x, wg, wu = (t.cuda().to(e4m3) for t in (x, wg, wu))
    _, s = hy.gated_ffn_fp8(x, sx.cuda(), wg, one, wu, one, act, fp8_out=True)
    ref = np.abs(op.act(act, g.astype(float))[0])
    tol = bounds(act, g.astype(float))[0] + 2 * N * ref  # the scale's division
    got = s.double().cpu().numpy() * 448
    assert (got == got[:, :1]).all()
    got = got[:, 0]
    kept = ref > 2.0 ** -99  # the scale's floor is 2^-100 / 448
    over = np.abs(got - ref) - tol
    assert kept.sum() > M / 2 and over[kept].max() <= 0, (g[kept][over[kept].argmax()], over[kept].max())
    assert (got[~kept] < 2.0 ** -98).all()


@pytest.mark.parametrize("act", list(K))
def test_slopes_of_small_values(act):
    """dg = act'(g) and du = act(g), rounded to bf16 once: the products by 1 and 0 leave them as they are."""
    import torch
    import hyena_long_convolution_b200 as hy
    M = 600
    g = gates(8 * M, 1).reshape(M, 8)
    one = torch.ones(M, 8, device="cuda")
    eye, none = torch.eye(8), torch.zeros(8, 8)
    wg, wu = (torch.cat(p, 1).to(torch.bfloat16).cuda() for p in ((eye, none), (none, eye)))  # dx = [dg | du]
    x = torch.zeros(M, 16, dtype=torch.bfloat16, device="cuda")
    dx = hy.gated_ffn_backward(one.bfloat16(), x, wg, wu, torch.from_numpy(g).cuda(), one, act).dx
    dx = dx.double().cpu().numpy()
    g = g.astype(float)
    for got, ref, tol, what in zip((dx[:, 8:], dx[:, :8]), op.act(act, g), bounds(act, g), ("du", "dg")):
        over = np.abs(got - ref) - (2.0 ** -8 * np.abs(ref) + 1.01 * tol + TINY)
        i = np.unravel_index(over.argmax(), over.shape)
        assert np.isfinite(got).all() and over[i] <= 0, (what, g[i], got[i], ref[i], tol[i])
