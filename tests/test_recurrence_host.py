"""Refusals of the gated recurrence's entry points, on the CPU: argument
checks run before any launch, so made-up addresses are never read."""
import pytest

import hyena_long_convolution_b200 as hy

INVALID, ALIGN, UNSUP, WORKSPACE = 1, 2, 3, 6
A = 1 << 20  # an aligned address
BIG = 1 << 40


def forward(**kw):
    a = dict(x1=A, x2=A, x3=A, ld_x=64, gate=A, ld_g=64, rate=A, ds=None, reset=None, norm=1, y=A, ld_y=64, si=None,
             so=None, us=None, B=1, L=100, D=64, ws=A, nb=BIG)
    a.update(kw)
    return hy.lib().hyena_gated_recurrence(*a.values(), None)


def backward(**kw):
    a = dict(dy=A, ld_dy=64, x1=A, x2=A, x3=A, ld_x=64, gate=A, ld_g=64, rate=A, ds=None, reset=None, norm=1, us=A,
             dso=None, dx1=A, dx2=A, dx3=A, ld_dx=64, dg=A, ld_dg=64, dr=A, dds=None, dsi=None, B=1, L=100, D=64,
             ws=A, nb=BIG)
    a.update(kw)
    return hy.lib().hyena_gated_recurrence_backward(*a.values(), None)


def decode(**kw):
    a = dict(x1=A, x2=A, x3=A, ld_x=64, gate=A, ld_g=64, rate=A, ds=None, norm=1, y=A, ld_y=64, s=A, B=1, D=64)
    a.update(kw)
    return hy.lib().hyena_gated_recurrence_decode(*a.values(), None)


COMMON = [(dict(x1=None), INVALID), (dict(gate=None), INVALID), (dict(rate=None), INVALID), (dict(B=0), INVALID),
          (dict(ld_x=56), INVALID), (dict(ld_g=56), INVALID), (dict(D=60), ALIGN), (dict(ld_x=68), ALIGN),
          (dict(ld_g=68), ALIGN), (dict(gate=A + 2), ALIGN), (dict(rate=A + 4), ALIGN), (dict(ds=A + 4), ALIGN)]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(L=-1), INVALID), (dict(y=None), INVALID), (dict(ld_y=68), ALIGN), (dict(si=A + 4), ALIGN),
    (dict(so=A + 8), ALIGN), (dict(us=A + 4), ALIGN), (dict(ws=None), WORKSPACE), (dict(nb=1000), WORKSPACE),
    (dict(ws=A + 8), ALIGN), (dict(L=2 ** 31 - 1, B=4096), UNSUP), (dict(L=2 ** 31 - 1, ld_x=2 ** 20), UNSUP),
    (dict(L=2 ** 31 - 1, ld_g=2 ** 20), UNSUP)])
def test_forward_refuses(kw, code):
    assert forward(**kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(dy=None), INVALID), (dict(us=None), INVALID), (dict(dr=None), INVALID), (dict(dx1=None), INVALID),
    (dict(dx2=None), INVALID), (dict(dx3=None), INVALID), (dict(dg=None), INVALID), (dict(ld_dy=56), INVALID),
    (dict(ld_dx=56), INVALID), (dict(ld_dg=56), INVALID), (dict(ld_dx=68), ALIGN), (dict(ld_dg=68), ALIGN),
    (dict(dx2=A + 2), ALIGN), (dict(dg=A + 2), ALIGN), (dict(us=A + 4), ALIGN), (dict(dso=A + 4), ALIGN),
    (dict(dsi=A + 4), ALIGN), (dict(dr=A + 4), ALIGN), (dict(dds=A + 4), ALIGN), (dict(ws=None), WORKSPACE),
    (dict(nb=1000), WORKSPACE), (dict(ws=A + 8), ALIGN)])
def test_backward_refuses(kw, code):
    assert backward(**kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(s=None), INVALID), (dict(s=A + 4), ALIGN), (dict(y=None), INVALID), (dict(ld_y=56), INVALID)])
def test_decode_refuses(kw, code):
    assert decode(**kw) == code


def test_workspace_size():
    size = hy.lib().hyena_gated_recurrence_workspace_size
    assert size(0, 10, 64) == size(1, -1, 64) == size(1, 10, 0) == size(1, 10, 60) == 0
    assert 0 < size(1, 0, 64) <= size(1, 64, 64) < size(1, 65, 64) < size(2, 65, 64) < size(2, 65, 72)


def test_binding_refuses():
    import torch
    bf = dict(dtype=torch.bfloat16)
    x = torch.zeros(2, 5, 64, **bf)
    lr = torch.zeros(64)
    with pytest.raises(ValueError, match="CUDA"):
        hy.gated_recurrence(x, x, x, x, lr)
    with pytest.raises(ValueError, match="CUDA"):
        hy.gated_recurrence_decode(x[:, 0], x[:, 0], x[:, 0], x[:, 0], lr, None, torch.zeros(2, 64))
    with pytest.raises(ValueError, match="CUDA"):
        hy.gated_recurrence_backward(x, x, x, x, x, lr, None, torch.zeros(2, 1, 64))
    with pytest.raises(ValueError, match="reset"):
        hy._reset(torch.zeros(2, 5), 2, 5)
    with pytest.raises(ValueError, match="reset"):
        hy._reset(torch.zeros(2, 4, dtype=torch.bool), 2, 5)
    with pytest.raises(ValueError, match="current"):
        hy._here(x)
