"""Of a product's workspace only the header has to be zero, and only that is
cleared: what lies behind it, 19 MB and for a gradient more, is written before it
is read."""
import re
import os

import pytest

import hyena_long_convolution_b200 as hy

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_header_size():
    text = open(os.path.join(ROOT, "include", "hyena.h")).read()
    assert int(re.search(r"#define HYENA_PRODUCT_HEADER (\d+)", text)[1]) == hy.PRODUCT_HEADER
    for M in (0, 1, 40, 5000):
        assert hy.lib().hyena_fp8_matmul_workspace_size(M, 64, 64) >= hy.PRODUCT_HEADER


def test_the_header_alone_is_cleared(monkeypatch):
    import torch
    taken = []

    class Lib:
        def __getattr__(self, name):
            if name == "hyena_modal_workspace_init":
                return lambda p, n, st: taken.append(n) or 0
            return getattr(real, name)
    real = hy.lib()
    monkeypatch.setattr(hy, "lib", lambda: Lib())
    monkeypatch.setattr(hy, "_stream", lambda s: None)
    empty = torch.empty
    sizes = []
    monkeypatch.setattr(torch, "empty", lambda n, dtype=None, device=None: sizes.append(n) or empty(16, dtype=dtype))
    hy.MatmulWorkspace(5000, 64, 64)
    hy.FfnWorkspace(5000, 64, 64, backward=True)
    assert taken == [hy.PRODUCT_HEADER] * 2
    assert sizes == [real.hyena_fp8_matmul_workspace_size(5000, 64, 64),
                     real.hyena_gated_ffn_workspace_size(5000, 64, 64, 1)]


def normal(*shape, seed, scale=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(torch.bfloat16).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("M,D,F", [(1, 264, 520), (20, 4400, 264), (40, 528, 1000), (100, 4400, 4880), (300, 4400, 3328),
                                   (300, 272, 520), (1000, 1040, 264)])
def test_rubbish_behind_the_header(M, D, F):
    """Whole tiles, and shared ones in 2 to 4 parts: the same bits whatever was there."""
    import torch
    x, wg, wu = normal(M, D, seed=1), normal(F, D, seed=2, scale=D ** -0.5), normal(F, D, seed=3, scale=D ** -0.5)
    dy, g, u = (normal(M, F, seed=s) for s in (4, 5, 6))
    q, s = hy.fp8_quantize(x)
    w = hy.fp8_quantize(wg, block=128)
    ws = hy.FfnWorkspace(M, D, F, backward=True)
    out = []
    for byte in (0, 0xff, 0x7f):  # NaN in bf16 and fp32; large numbers
        ws.buf[hy.PRODUCT_HEADER:] = byte
        out.append([hy.fp8_matmul(q, s, *w, workspace=ws), hy.gated_ffn(x, wg, wu, workspace=ws),
                    hy.gated_ffn_fp8(q, s, *w, *w, workspace=ws),
                    *hy.gated_ffn_backward(dy, x, wg, wu, g, u, workspace=ws)])
    for other in out[1:]:
        for a, b in zip(out[0], other):
            assert torch.isfinite(a.float()).all() and torch.equal(a, b)
    hy.workspace_check(ws)
