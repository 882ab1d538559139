"""Refusals of the 8-bit products' and the feed-forward block's entry points, on
the CPU: argument checks run before any launch, so made-up addresses are never
read."""
import pytest

import hyena_long_convolution_b200 as hy

INVALID, ALIGN, UNSUP, WORKSPACE = 1, 2, 3, 6
BF16, F32 = 1, 2
A = 1 << 20  # an aligned address
BIG = 1 << 62


def quantize(**kw):
    a = dict(x=A, ld_x=64, xt=BF16, q=A, ld_q=64, s=A, block=1, M=3, D=64)
    a.update(kw)
    return hy.lib().hyena_fp8_quantize(*a.values(), None)


def matmul(**kw):
    a = dict(x=A, ld_x=64, sx=A, group=128, w=A, ld_w=64, sw=A, y=A, ld_y=32, yt=BF16, M=3, N=32, K=64, ws=A, nb=BIG)
    a.update(kw)
    return hy.lib().hyena_fp8_matmul(*a.values(), None)


def ffn(**kw):
    a = dict(x=A, ld_x=64, wg=A, wu=A, ld_w=64, act=1, y=A, ld_y=32, g=A, u=A, ld_g=32, kt=F32, M=3, D=64, F=32, ws=A,
             nb=BIG)
    a.update(kw)
    return hy.lib().hyena_gated_ffn(*a.values(), None)


def ffn_fp8(**kw):
    a = dict(x=A, ld_x=64, sx=A, group=0, wg=A, sg=A, wu=A, su=A, ld_w=64, act=1, y=None, ld_y=0, q=A, ld_q=32, s=A,
             M=3, D=64, F=32, ws=A, nb=BIG)
    a.update(kw)
    return hy.lib().hyena_gated_ffn_fp8(*a.values(), None)


def backward(**kw):
    a = dict(dy=A, ld_dy=32, x=A, ld_x=64, wg=A, wu=A, ld_w=64, g=A, u=A, ld_g=32, kt=F32, act=1, dx=A, ld_dx=64,
             dwg=A, dwu=A, ld_dw=64, M=3, D=64, F=32, ws=A, nb=BIG)
    a.update(kw)
    return hy.lib().hyena_gated_ffn_backward(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(D=0), INVALID), (dict(D=60), ALIGN), (dict(M=1 << 31), UNSUP),
    (dict(D=(1 << 20) + 8), UNSUP), (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID),
    (dict(x=A + 8), ALIGN), (dict(q=A + 8), ALIGN), (dict(s=A + 2), ALIGN), (dict(ld_x=56), INVALID),
    (dict(ld_q=56), INVALID), (dict(ld_x=68), ALIGN), (dict(ld_q=68), ALIGN), (dict(xt=0), INVALID),
    (dict(xt=3), INVALID), (dict(block=0), INVALID), (dict(block=64), UNSUP), (dict(ld_x=1 << 40), UNSUP)])
def test_quantize_refuses(kw, code):
    assert quantize(**kw) == code


SIZES = [(dict(M=-1), INVALID), (dict(M=1 << 31), UNSUP), (dict(ws=None), WORKSPACE), (dict(nb=16), WORKSPACE),
         (dict(ws=A + 8), ALIGN), (dict(x=None), INVALID), (dict(x=A + 8), ALIGN), (dict(ld_x=56), INVALID),
         (dict(ld_x=68), ALIGN), (dict(ld_w=56), INVALID), (dict(ld_w=68), ALIGN), (dict(ld_w=1 << 40), UNSUP)]


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(N=28), ALIGN), (dict(K=60), ALIGN), (dict(K=(1 << 20) + 8), UNSUP),
    (dict(ld_x=72), ALIGN), (dict(ld_w=72), ALIGN), (dict(ld_y=24), INVALID), (dict(ld_y=36), ALIGN),
    (dict(w=None), INVALID), (dict(w=A + 8), ALIGN), (dict(y=None), INVALID), (dict(y=A + 8), ALIGN),
    (dict(sx=None), INVALID), (dict(sx=A + 1), ALIGN), (dict(sw=None), INVALID), (dict(sw=A + 2), ALIGN),
    (dict(group=-1), INVALID), (dict(group=64), UNSUP), (dict(yt=0), INVALID), (dict(yt=3), INVALID)])
def test_matmul_refuses(kw, code):
    assert matmul(**kw) == code


FFN = [(dict(D=0), INVALID), (dict(F=0), INVALID), (dict(D=60), ALIGN), (dict(F=28), ALIGN),
       (dict(F=(1 << 20) + 8), UNSUP), (dict(act=0), INVALID), (dict(act=5), INVALID), (dict(wg=None), INVALID),
       (dict(wu=None), INVALID), (dict(wg=A + 8), ALIGN), (dict(wu=A + 8), ALIGN)]


@pytest.mark.parametrize("kw,code", SIZES + FFN + [
    (dict(y=None), INVALID), (dict(y=A + 2), ALIGN), (dict(ld_y=24), INVALID), (dict(ld_y=36), ALIGN),
    (dict(g=None), INVALID), (dict(u=None), INVALID), (dict(g=A + 4), ALIGN), (dict(ld_g=24), INVALID),
    (dict(ld_g=36), ALIGN), (dict(kt=0), INVALID)])
def test_ffn_refuses(kw, code):
    assert ffn(**kw) == code


@pytest.mark.parametrize("kw,code", SIZES + FFN + [
    (dict(y=A, ld_y=32), INVALID), (dict(q=None), INVALID), (dict(q=A + 8), ALIGN), (dict(ld_q=24), INVALID),
    (dict(ld_q=40), ALIGN), (dict(s=None), INVALID), (dict(s=A + 2), ALIGN), (dict(q=None, y=A, ld_y=24), INVALID),
    (dict(q=None, y=A + 2, ld_y=32), ALIGN), (dict(sx=None), INVALID), (dict(sg=None), INVALID),
    (dict(su=None), INVALID), (dict(su=A + 2), ALIGN), (dict(group=64), UNSUP), (dict(ld_x=72), ALIGN)])
def test_ffn_fp8_refuses(kw, code):
    assert ffn_fp8(**kw) == code


@pytest.mark.parametrize("kw,code", SIZES + FFN + [
    (dict(dy=None), INVALID), (dict(dy=A + 2), ALIGN), (dict(ld_dy=24), INVALID), (dict(g=None), INVALID),
    (dict(u=None), INVALID), (dict(u=A + 8), ALIGN), (dict(ld_g=24), INVALID), (dict(kt=0), INVALID),
    (dict(kt=3), INVALID), (dict(dx=None), INVALID), (dict(dx=A + 2), ALIGN), (dict(ld_dx=56), INVALID),
    (dict(ld_dx=68), ALIGN), (dict(dwg=None), INVALID), (dict(dwu=None), INVALID), (dict(dwu=A + 2), ALIGN),
    (dict(ld_dw=56), INVALID), (dict(ld_dw=68), ALIGN)])
def test_backward_refuses(kw, code):
    assert backward(**kw) == code


@pytest.mark.parametrize("call,outs,ins", [
    (quantize, ("q", "s"), ("x",)), (matmul, ("y",), ("x", "w", "sx", "sw", "ws")),
    (ffn, ("y", "g", "u"), ("x", "wg", "wu", "ws")), (ffn_fp8, ("q", "s"), ("x", "sx", "wg", "sg", "wu", "su", "ws")),
    (backward, ("dx", "dwg", "dwu"), ("dy", "x", "wg", "wu", "g", "u", "ws"))])
def test_an_output_in_place_of_another_argument_is_refused(call, outs, ins):
    import itertools
    names = outs + ins
    apart = {n: A + i * (1 << 20) for i, n in enumerate(names)}
    for out, other in itertools.product(outs, names):
        if out != other:
            assert call(**{**apart, out: apart[other]}) == INVALID, (out, other)


def test_no_rows_launch_nothing():
    assert quantize(M=0, x=None, q=None, s=None) == 0
    assert matmul(M=0, x=None, sx=None, y=None, ws=None) == 0
    assert ffn(M=0, x=None, y=None, g=None, u=None, ws=None) == 0
    assert ffn_fp8(M=0, x=None, sx=None, q=None, s=None, ws=None) == 0
    assert hy.last_launch_count() == 0


def test_workspace_size():
    m, f = hy.lib().hyena_fp8_matmul_workspace_size, hy.lib().hyena_gated_ffn_workspace_size
    assert m(-1, 32, 64) == m(3, 0, 64) == m(3, 32, 60) == f(-1, 64, 32, 0) == f(3, 60, 32, 1) == 0
    rows = (0, 1, 2, 16, 17, 33, 64, 65, 128, 129, 200, 256, 257, 1000, 8192, 100000)
    for N, K in ((32, 64), (4096, 11008), (12288, 4096), (8, 8), (1032, 1040)):
        sizes = [m(M, N, K) for M in rows]  # one for many rows serves fewer
        assert sizes == sorted(sizes) and 0 < sizes[0] and sizes[-1] < 64 << 20
        for back in (0, 1):
            sizes = [f(M, K, N, back) for M in rows]
            assert sizes == sorted(sizes) and 0 < sizes[0]
            assert sizes[-1] < (64 << 20) + back * (256 << 20) + back * 100000 * N * 4


def test_binding_refuses():
    import torch
    x = torch.zeros(3, 64, dtype=torch.bfloat16)
    q, s1 = torch.zeros(3, 64, dtype=torch.float8_e4m3fn), torch.ones(3, 1)
    w, wq, sw = torch.zeros(32, 64, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.float8_e4m3fn), torch.ones(1, 1)
    g = torch.zeros(3, 32)
    calls = [lambda: hy.fp8_quantize(x), lambda: hy.fp8_matmul(q, s1, wq, sw), lambda: hy.gated_ffn(x, w, w),
             lambda: hy.gated_ffn_fp8(q, s1, wq, sw, wq, sw),
             lambda: hy.gated_ffn_backward(x[:, :32], x, w, w, g, g)]
    for f in calls:
        with pytest.raises(ValueError, match="CUDA"):
            f()
    bad = [(lambda: hy.fp8_quantize(x, block=64), "block"), (lambda: hy.fp8_quantize(q), "x must"),
           (lambda: hy.fp8_matmul(x, s1, wq, sw), "x must"), (lambda: hy.fp8_matmul(q, s1[:2], wq, sw), "scales"),
           (lambda: hy.fp8_matmul(q, s1, wq[:, :32], sw), "weight"), (lambda: hy.fp8_matmul(q, s1, w, sw), "weight"),
           (lambda: hy.fp8_matmul(q, s1, wq, torch.ones(2, 1)), "weight_scales"),
           (lambda: hy.gated_ffn(x, w, w, "relu"), "activation"), (lambda: hy.gated_ffn(x, w, w[:16]), "up_weight"),
           (lambda: hy.gated_ffn(x, wq, wq), "bf16"), (lambda: hy.gated_ffn(x[:, :32], w, w), "weights"),
           (lambda: hy.gated_ffn_fp8(q, s1, w, sw, w, sw), "e4m3"),
           (lambda: hy.gated_ffn_fp8(q, s1, wq, sw, wq, torch.ones(1)), "up_scales"),
           (lambda: hy.gated_ffn_backward(x, x, w, w, g, g), "dy"),
           (lambda: hy.gated_ffn_backward(x[:, :32], x, w, w, g, None), "both"),
           (lambda: hy.gated_ffn_backward(x[:, :32], x, w, w, g, g.bfloat16()), "type")]
    for f, match in bad:
        with pytest.raises(ValueError, match=match):
            f()
