"""The norm's gradient where each CTA goes through many more rows than its ring
of stages holds, so that every stage is asked for again, several times over and
with a last round that is not full; and the 8-bit norm with all that it can
write.  Against the fp64 oracle with the bounds of test_parity_norm."""
import numpy as np
import pytest

from oracle import norm as onorm

from .test_parity_norm import EPS, N, check_fp8, f64, make, near

pytestmark = pytest.mark.gpu


# Rows a CTA: 5 to 15, by 2368 CTAs at 264 channels, 1184 at 520, 592 at 1032, 296 at 4096 and 8192, 148 above;
# stages: 2 (fp32 at 4096, both at 8192, 16384) to 6.  Above 10240 channels an fp32 dresidual_out does not go
# through the ring.
@pytest.mark.parametrize("M,D,res", [
    (30011, 264, "bf16"), (15013, 520, "fp32"), (9001, 1032, "bf16"), (6001, 1032, "fp32"), (2501, 4096, None),
    (2501, 4096, "bf16"), (1511, 4096, "fp32"), (1301, 8192, "bf16"), (1301, 8192, "fp32"), (1499, 8200, "bf16"),
    (701, 8200, "fp32"), (701, 10248, "fp32"), (1001, 16384, "bf16"), (701, 16384, "fp32")])
def test_gradient(M, D, res):
    import torch
    import hyena_long_convolution_b200 as hy
    x, r, w, dy, dho, h = make(M, D, M + D, res)
    c = [t.cuda() for t in (h, w, dy, dho)]
    rstd = torch.from_numpy(onorm.rstd(f64(h), EPS)).float().cuda()
    for with_dho in (False, True):
        g = hy.rms_norm_backward(c[2], c[0], c[1], rstd, dresidual_out=c[3] if with_dho else None)
        dh, dw, sc, scw = onorm.backward(f64(dy), f64(h), f64(w), EPS, f64(dho) if with_dho else None)
        near(g.dx, dh, 200 * N * sc, "dx", 2.0 ** -8)
        near(g.dweight, dw, (40 + M) * N * scw, "dweight")
        if res == "fp32":
            near(g.dresidual, dh, 200 * N * sc, "dresidual")
    g2 = hy.rms_norm_backward(c[2], c[0], c[1], rstd, dresidual_out=c[3])
    assert all(a is b or torch.equal(a, b) for a, b in zip(g2, g))


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("M,D,res", [(5, 72, "bf16"), (301, 264, "fp32"), (33, 1032, "bf16"), (7, 4096, "fp32"),
                                     (700, 128, "bf16"), (3, 16384, "fp32"), (9, 520, None)])
def test_8_bit_norm_writes_all_its_outputs(M, D, res, group):
    import torch
    import hyena_long_convolution_b200 as hy
    x, r, w, dy, dho, h = make(M, D, M * D, res, "bf16")
    ho = None if r is None else torch.empty_like(r, device="cuda")
    rstd = torch.empty(M, device="cuda")
    rc = None if r is None else r.cuda()
    q = torch.zeros(M, D, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(M, 1 if group == 0 else -(-D // 128), device="cuda")
    out = hy.rms_norm_fp8(x.cuda(), w.cuda(), EPS, residual=rc, residual_out=ho, group=group, q=q, scales=s, rstd=rstd)
    assert out[0] is q and out[1] is s
    check_fp8(q, s, h, w, group)
    want = onorm.rstd(f64(h), EPS)
    near(rstd, want, 30 * N * want, "rstd")
    if r is not None:
        assert torch.equal(ho.cpu(), h)
        hy.rms_norm_fp8(x.cuda(), w.cuda(), EPS, residual=rc, residual_out=rc, group=group)  # in place
        assert torch.equal(rc, ho)
