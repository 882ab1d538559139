"""Refusals of the norm's entry points, on the CPU: argument checks run before
any launch, so made-up addresses are never read."""
import pytest

import hyena_long_convolution_b200 as hy

INVALID, ALIGN, UNSUP, WORKSPACE = 1, 2, 3, 6
BF16, F32 = 1, 2
A = 1 << 20  # an aligned address


def norm(**kw):
    a = dict(x=A, ld_x=64, r=A, ro=A, ld_r=64, rt=BF16, w=A, wt=F32, eps=1e-6, y=A, ld_y=64, rstd=None, M=3, D=64)
    a.update(kw)
    return hy.lib().hyena_rms_norm(*a.values(), None)


def fp8(**kw):
    a = dict(x=A, ld_x=64, r=A, ro=A, ld_r=64, rt=BF16, w=A, wt=F32, eps=1e-6, y=A, ld_y=64, s=A, group=0, rstd=None,
             M=3, D=64)
    a.update(kw)
    return hy.lib().hyena_rms_norm_fp8(*a.values(), None)


def backward(**kw):
    a = dict(y=A, ld_y=64, h=A, ld_h=64, ht=F32, w=A, wt=F32, rstd=A, dro=A, ld_r=64, dx=A, ld_x=64, dr=A, ld_dr=64,
             dw=A, M=3, D=64, ws=A, nb=1 << 30)
    a.update(kw)
    return hy.lib().hyena_rms_norm_backward(*a.values(), None)


COMMON = [(dict(M=-1), INVALID), (dict(D=0), INVALID), (dict(D=60), ALIGN), (dict(w=None), INVALID),
          (dict(D=16392, ld_x=16392, ld_y=16392, ld_r=16392), UNSUP), (dict(M=1 << 31), UNSUP),
          (dict(ld_x=56), INVALID), (dict(ld_y=56), INVALID), (dict(ld_r=56), INVALID), (dict(ld_x=68), ALIGN),
          (dict(ld_r=68), ALIGN), (dict(ld_y=68), ALIGN), (dict(wt=0), INVALID), (dict(wt=3), INVALID),
          (dict(w=A + 4), ALIGN), (dict(y=None), INVALID), (dict(y=A + 8), ALIGN), (dict(rstd=A + 4), ALIGN)]
FORWARD = COMMON + [(dict(x=None), INVALID), (dict(x=A + 2), ALIGN), (dict(rt=0), INVALID), (dict(rt=7), INVALID),
                    (dict(r=None), INVALID), (dict(ro=A + 4), ALIGN), (dict(eps=-1.0), INVALID),
                    (dict(eps=float("nan")), INVALID)]


@pytest.mark.parametrize("kw,code", FORWARD)
def test_norm_refuses(kw, code):
    assert norm(**kw) == code


@pytest.mark.parametrize("kw,code", FORWARD + [(dict(s=None), INVALID), (dict(s=A + 4), ALIGN),
                                               (dict(group=-1), INVALID), (dict(group=64), UNSUP)])
def test_fp8_refuses(kw, code):
    assert fp8(**kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(h=None), INVALID), (dict(ht=0), INVALID), (dict(ht=BF16), INVALID), (dict(dw=None), INVALID),
    (dict(rstd=None), INVALID), (dict(ld_h=56), INVALID), (dict(ld_dr=56), INVALID), (dict(ld_dr=68), ALIGN),
    (dict(dr=A + 4), ALIGN), (dict(dw=A + 4), ALIGN), (dict(ws=None), WORKSPACE), (dict(nb=64), WORKSPACE),
    (dict(ws=A + 4), ALIGN)])
def test_backward_refuses(kw, code):
    assert backward(**kw) == code


def test_no_rows_launch_nothing():
    assert norm(M=0, x=None, y=None) == 0 and fp8(M=0, x=None, y=None, s=None) == 0


def test_workspace_size():
    size = hy.lib().hyena_rms_norm_backward_workspace_size
    assert size(-1, 64) == size(3, 0) == size(3, 60) == size(3, 16392) == 0
    assert 0 < size(0, 64) <= size(1, 64) <= size(3, 64) < size(3, 72)


def test_binding_refuses():
    import torch
    x = torch.zeros(3, 64, dtype=torch.bfloat16)
    w = torch.ones(64)
    for f in (hy.rms_norm, hy.rms_norm_fp8):
        with pytest.raises(ValueError, match="CUDA"):
            f(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        hy.rms_norm_backward(x, x, w, torch.ones(3))
    u8 = torch.zeros(1024, dtype=torch.uint8)
    for work in (u8[::2], u8[:1].expand(99), torch.zeros(1024)):
        with pytest.raises(ValueError, match="workspace"):
            hy.rms_norm_backward(x, x, w, torch.ones(3), workspace=work)
