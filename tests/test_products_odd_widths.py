"""Codes of widths that are no multiples of 16 from each call that allocates them
to each that reads them: the products want row strides that are."""
import numpy as np
import pytest

from oracle import products as op

pytestmark = pytest.mark.gpu

N = 2.0 ** -24


def f64(t):
    return t.double().cpu().numpy()


def values(q, s, block=1):
    return op.values(f64(q).reshape(-1, q.shape[-1]), f64(s), block)


def product_is_right(y, x, w):
    """Sums over each 128 of K and then over the groups, by additions that may cut off, and y's rounding."""
    ref, size = x @ w.T, np.abs(x) @ np.abs(w).T
    K = x.shape[1]
    assert (np.abs(f64(y).reshape(ref.shape) - ref) <= 2 * N * (128 + K / 128 + 8) * size + 2.0 ** -8 * np.abs(ref)).all()


@pytest.mark.parametrize("D,F", [(8, 8), (1032, 520), (264, 1000), (520, 136), (16, 24)])
@pytest.mark.parametrize("rows", [(1,), (3,), (300,), (2, 1), (2, 70), (1, 5), (0,)])
def test_codes_from_call_to_call(rows, D, F):
    import torch
    import hyena_long_convolution_b200 as hy
    g = torch.Generator().manual_seed(D + len(rows))
    x = torch.randn(*rows, D, generator=g).to(torch.bfloat16).cuda()
    weights = [(torch.randn(n, d, generator=g) * d ** -0.5).to(torch.bfloat16).cuda()
               for n, d in ((D, D), (F, D), (F, D), (D, F))]
    W = [hy.fp8_quantize(w, block=128) for w in weights]
    V = [values(*w, 128) for w in W]
    M = int(np.prod(rows))
    norm = hy.rms_norm_fp8(x, torch.ones(D, device="cuda"), group=128)
    whole = hy.rms_norm_fp8(x, torch.ones(D, device="cuda"))
    for q, s in (norm, whole, hy.fp8_quantize(x)):
        assert q.shape == x.shape
        y = hy.fp8_matmul(q, s, *W[0])
        assert y.shape == (*rows, D)
        product_is_right(y, values(q, s), V[0])
    block = hy.gated_ffn_fp8(*norm, *W[1], *W[2], "silu")
    q, s = hy.gated_ffn_fp8(*norm, *W[1], *W[2], "silu", fp8_out=True)
    assert q.shape == (*rows, F) and s.shape == (M, -(-F // 128))
    # y's own rounding (2^-8), the code's (2^-4, or 2^-10 of a scale) and the sums' (by the bound
    # of the products, for unit-sized sums less than 2^-8 too)
    each = op.spread(f64(s), 1, (M, F)) if M else np.zeros((0, F))
    yb = f64(block).reshape(M, F)
    assert (np.abs(values(q, s) - yb) <= 2.0 ** -4 * np.abs(yb) * 1.02 + 2.0 ** -8 * np.abs(yb) + 2.0 ** -10 * each).all()
    down = hy.fp8_matmul(q, s, *W[3])
    assert down.shape == x.shape
    product_is_right(down, values(q, s), V[3])


def test_one_row_of_given_codes():
    """With one row there is no stride to object to."""
    import torch
    import hyena_long_convolution_b200 as hy
    x = torch.ones(1, 24, dtype=torch.bfloat16, device="cuda")
    w = hy.fp8_quantize(torch.ones(24, 24, dtype=torch.bfloat16, device="cuda"), block=128)
    q = torch.zeros(1, 24, device="cuda").to(torch.float8_e4m3fn)
    got = hy.gated_ffn_fp8(*hy.fp8_quantize(x), *w, *w, "identity", fp8_out=True, q=q)
    assert got[0] is q and (q.float() == 448.0).all() and abs(got[1].item() * 448 / 576 - 1) < 4 * 8 * N


def test_widths_of_whole_16_stay_contiguous():
    import torch
    import hyena_long_convolution_b200 as hy
    x = torch.ones(3, 5, 48, dtype=torch.bfloat16, device="cuda")
    assert hy.fp8_quantize(x)[0].is_contiguous()
    assert hy.rms_norm_fp8(x, torch.ones(48, device="cuda"))[0].is_contiguous()
