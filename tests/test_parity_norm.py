"""The RMS norm (bf16 and e4m3 outputs, gradient) against its fp64 oracle,
with tolerances that follow from the kernels' arithmetic.

With n = 2^-24 (half a step of fp32): the sum of squares is at most 32 FMAs a
thread, 5 butterfly steps and 16 warps' sums, all of one sign: 53 n relative;
the mean, eps and the root: 30 n for rstd; y = h rstd weight: 33 n.  A scale:
34 n more by its division, y / scale 70 n in all.  The gradient's dot product
adds 53 n of the sum of its terms' absolute values and each factor 35 n, dh
below 200 n of the absolute terms.  dweight: 40 n and one step a row.
Outputs add half a step of their type: bf16 2^-8, e4m3 2^-4 of the value or
2^-10 among its subnormals.
"""
import numpy as np
import pytest

from oracle import norm as onorm

pytestmark = pytest.mark.gpu

N = 2.0 ** -24
EPS = 1e-5


def make(M, D, seed, res, weight="fp32", scale=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32, None: torch.bfloat16}
    x = (scale * torch.randn(M, D, generator=g)).to(torch.bfloat16)
    r = None if res is None else (3.0 * scale * torch.randn(M, D, generator=g)).to(dt[res])
    w = (1.0 + 0.3 * torch.randn(D, generator=g)).to(dt[weight])
    dy = torch.randn(M, D, generator=g).to(torch.bfloat16)
    dho = torch.randn(M, D, generator=g).to(dt[res])
    h = x if r is None else (x.float() + r.float()).to(r.dtype)
    return x, r, w, dy, dho, h


def f64(t):
    return t.double().cpu().numpy()


def near(got, ref, tol, what, half=0.0):
    got = f64(got)
    assert got.shape == ref.shape and np.isfinite(got).all(), what
    over = np.abs(got - ref) - (tol + half * np.abs(ref) + 1e-30)
    assert over.max() <= 0, f"{what}: over by {over.max():.3e}"


def check_fp8(q, s, h, w, group):
    y = onorm.forward(f64(h), f64(w), EPS)
    ref = onorm.scales(y, group)
    near(s, ref, 34 * N * ref, "scales")
    each = ref if group == 0 else np.repeat(ref, group, 1)[:, :y.shape[1]]
    z = y / each
    near(q.float(), z, 70 * N * np.abs(z) + 2.0 ** -10, "q", 2.0 ** -4)


@pytest.mark.parametrize("weight", ["fp32", "bf16"])
@pytest.mark.parametrize("res", [None, "bf16", "fp32"])
@pytest.mark.parametrize("M,D", [(1, 8), (3, 64), (2, 72), (33, 128), (5, 136), (1, 256), (2, 264), (7, 1032),
                                 (1, 2048), (2, 2056), (3, 4096), (2, 8200), (1, 16384), (601, 40),
                                 (30001, 64), (15001, 128), (7501, 200), (1301, 512), (1301, 1000)])
def test_matches_oracle(M, D, res, weight):
    import torch
    import hyena_long_convolution_b200 as hy
    x, r, w, dy, dho, h = make(M, D, M + D, res, weight)
    c = [None if t is None else t.cuda() for t in (x, r, w, dy, dho, h)]
    ho = None if r is None else torch.empty_like(c[1])
    rstd = torch.empty(M, device="cuda")
    y = hy.rms_norm(c[0], c[2], EPS, residual=c[1], residual_out=ho, rstd=rstd)
    if r is not None:
        assert torch.equal(ho, c[5])
    hd, wd = f64(h), f64(w)
    ref = onorm.forward(hd, wd, EPS)
    near(rstd, onorm.rstd(hd, EPS), 30 * N * onorm.rstd(hd, EPS), "rstd")
    near(y, ref, 33 * N * np.abs(ref), "y", 2.0 ** -8)
    for group in (0, 128):
        q, s = hy.rms_norm_fp8(c[0], c[2], EPS, residual=c[1], group=group)
        check_fp8(q, s, h, w, group)
    hg = c[0] if r is None else ho
    for with_dho in (False, True):
        g = hy.rms_norm_backward(c[3], hg, c[2], rstd, dresidual_out=c[4] if with_dho else None)
        dh, dw, sc, scw = onorm.backward(f64(dy), hd, wd, EPS, f64(dho) if with_dho else None)
        near(g.dx, dh, 200 * N * sc, "dx", 2.0 ** -8)
        near(g.dweight, dw, (40 + M) * N * scw, "dweight")
        if res == "fp32":
            near(g.dresidual, dh, 200 * N * sc, "dresidual")
        else:
            assert g.dresidual is g.dx


def test_views_batches_and_padding():
    """[B, L, D] tensors, row strides above D, residual_out in place; what lies
    between the rows stays as it was."""
    import torch
    import hyena_long_convolution_b200 as hy
    B, L, D, pad = 2, 5, 72, 8
    x, r, w, dy, dho, h = (None if t is None else t.cuda() for t in make(B * L, D, 4, "fp32"))
    rstd = torch.empty(B * L, device="cuda")
    ho = torch.empty_like(r)
    y = hy.rms_norm(x, w, EPS, residual=r, residual_out=ho, rstd=rstd)
    q, s = hy.rms_norm_fp8(x, w, EPS, residual=r, group=128)
    g = hy.rms_norm_backward(dy, ho, w, rstd, dresidual_out=dho)

    def padded(t, fill=9.0):
        p = torch.full((B, L, D + pad), fill, device="cuda").to(t.dtype)
        p[..., :D] = t.view(B, L, D)
        return p
    xp, rp, dyp, dp = padded(x), padded(r), padded(dy), padded(dho)
    yp, qp = padded(torch.zeros_like(x)), padded(torch.zeros_like(x)).to(torch.float8_e4m3fn)
    y2 = hy.rms_norm(xp[..., :D], w, EPS, residual=rp[..., :D], residual_out=rp[..., :D], y=yp[..., :D])
    assert torch.equal(y2, y.view(B, L, D)) and torch.equal(rp[..., :D], ho.view(B, L, D))
    q2, s2 = hy.rms_norm_fp8(xp[..., :D], w, EPS, residual=padded(r)[..., :D], group=128, q=qp[..., :D])
    assert torch.equal(q2.float(), q.view(B, L, D).float()) and torch.equal(s2, s)
    dxp = padded(torch.zeros_like(x))
    g2 = hy.rms_norm_backward(dyp[..., :D], rp[..., :D], w, rstd, dresidual_out=dp[..., :D], dresidual=dp[..., :D],
                              dx=dxp[..., :D])
    assert torch.equal(g2.dx, g.dx.view(B, L, D)) and torch.equal(g2.dweight, g.dweight)
    assert torch.equal(g2.dresidual, g.dresidual.view(B, L, D))
    for p in (xp, rp, dyp, dp, yp, dxp, qp.float()):
        assert (p[..., D:] == 9.0).all()


def test_zero_rows_tiny_rows_and_rows_not_finite():
    import torch
    import hyena_long_convolution_b200 as hy
    M, D = 6, 264
    x, _, w, dy, _, _ = (None if t is None else t.cuda() for t in make(M, D, 8, None))
    x[0] = 0.0
    x[1] = 1e-38
    x[2, 5] = float("nan")
    x[3, 200] = float("inf")
    x[4] = 0.0
    x[4, 7] = 3.0
    for group in (0, 128):
        q, s = hy.rms_norm_fp8(x, w, EPS, group=group)
        assert (q[0].float() == 0).all() and (s[0] > 0).all() and torch.isfinite(s[0]).all()
        assert torch.isfinite(q[[0, 1, 4, 5]].float()).all() and torch.isfinite(s[[0, 1, 4, 5]]).all()
        assert q[4, 7].float().abs() == 448.0
        assert torch.isnan(q[2].float()).all() and torch.isnan(s[2]).all()
        assert torch.isnan(q[3, 200].float()) and torch.isnan(s[3, -1 if group == 0 else 1])
        clean, sc = hy.rms_norm_fp8(x[[0, 1, 4, 5]], w, EPS, group=group)
        assert torch.equal(clean.float(), q[[0, 1, 4, 5]].float()) and torch.equal(sc, s[[0, 1, 4, 5]])
    rstd = torch.empty(M, device="cuda")
    y = hy.rms_norm(x, w, EPS, rstd=rstd)
    assert torch.isnan(y[2]).all() and torch.isfinite(y[[0, 1, 4, 5]]).all() and (y[0] == 0).all()
    g = hy.rms_norm_backward(dy, x, w, rstd)
    assert torch.isfinite(g.dx[[0, 1, 4, 5]]).all()


def test_no_rows():
    import torch
    import hyena_long_convolution_b200 as hy
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    assert hy.rms_norm(x, w).shape == (0, 64)
    q, s = hy.rms_norm_fp8(x, w, group=128)
    assert q.shape == (0, 64) and s.shape == (0, 1)
    g = hy.rms_norm_backward(x, x, w, torch.empty(0, device="cuda"))
    assert g.dx.shape == (0, 64) and (g.dweight == 0).all()


def test_other_stream_and_graph_replay():
    import torch
    import hyena_long_convolution_b200 as hy
    x, r, w, dy, dho, h = (t.cuda() for t in make(700, 1032, 9, "bf16"))
    rstd = torch.empty(700, device="cuda")
    ho = torch.empty_like(r)

    def all_of():
        y = hy.rms_norm(x, w, EPS, residual=r, residual_out=ho, rstd=rstd)
        q, s = hy.rms_norm_fp8(x, w, EPS, residual=r)
        g = hy.rms_norm_backward(dy, ho, w, rstd, dresidual_out=dho)
        return y, q.float(), s, g.dx, g.dweight
    ref = all_of()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = all_of()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    # the stream given instead of made current
    for st in (side, side.cuda_stream):
        y = hy.rms_norm(x, w, EPS, residual=r, residual_out=ho, rstd=rstd, stream=st)
        q, s = hy.rms_norm_fp8(x, w, EPS, residual=r, stream=st)
        g = hy.rms_norm_backward(dy, ho, w, rstd, dresidual_out=dho, stream=st)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, (y, q.float(), s, g.dx, g.dweight)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_of()
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, got))
    del graph


def test_a_block_from_the_residual_stream_to_its_gradient():
    """Norm, projection, recurrence, projection, norm as a layer runs them, and
    back; and the same layer token by token.  Against fp64 with the roundings
    between the calls left out: five bf16 roundings in a row of values that
    are summed with random signs, each 2^-8 at most."""
    import torch
    import hyena_long_convolution_b200 as hy
    torch.manual_seed(0)
    B, L, D = 2, 100, 128
    dev = dict(device="cuda")
    res = torch.randn(B, L, D, **dev)
    x = torch.randn(B, L, D, **dev).to(torch.bfloat16)
    w1, w2 = 1 + 0.1 * torch.randn(D, **dev), 1 + 0.1 * torch.randn(D, **dev)
    Win = (torch.randn(D, 4 * D, **dev) / D ** 0.5).to(torch.bfloat16)
    Wout = (torch.randn(D, D, **dev) / D ** 0.5).to(torch.bfloat16)
    lr = -torch.exp(torch.rand(D, **dev) * 6.9 - 6.9)
    dsk = torch.randn(D, **dev)
    dout = torch.randn(B, L, D, **dev).to(torch.bfloat16)

    h1, r1 = torch.empty_like(res), torch.empty(B * L, **dev)
    n1 = hy.rms_norm(x, w1, residual=res, residual_out=h1, rstd=r1)
    p = n1 @ Win
    parts = [p[:, :, i * D:(i + 1) * D] for i in range(4)]
    units = hy.recurrence_unit_states(B, L, D)
    S = torch.empty(B, D, **dev)
    y = hy.gated_recurrence(*parts, lr, dsk, unit_states=units, state_out=S)
    o = y @ Wout
    h2, r2 = torch.empty_like(res), torch.empty(B * L, **dev)
    n2 = hy.rms_norm(o, w2, residual=h1, residual_out=h2, rstd=r2)

    g2 = hy.rms_norm_backward(dout, h2, w2, r2)
    dy = g2.dx @ Wout.T
    dp = torch.empty_like(p)
    dparts = [dp[:, :, i * D:(i + 1) * D] for i in range(4)]
    gr = hy.gated_recurrence_backward(dy, *parts, lr, dsk, units, dx1=dparts[0], dx2=dparts[1], dx3=dparts[2],
                                      dgate=dparts[3])
    g1 = hy.rms_norm_backward(dp @ Win.T, h1, w1, r1, dresidual_out=g2.dresidual)

    leaf = {k: v.double().requires_grad_() for k, v in dict(res=res, x=x, w1=w1, w2=w2, lr=lr, dsk=dsk, Win=Win,
                                                             Wout=Wout).items()}

    def norm(h, w):
        return h * w / (h.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()
    hh = leaf["x"] + leaf["res"]
    a1, a2, a3, ag = (norm(hh, leaf["w1"]) @ leaf["Win"]).split(D, -1)
    l = leaf["lr"] * torch.sigmoid(ag)
    v = a1 * a2
    u, a = (-torch.expm1(2 * l)).sqrt() * v, l.exp()
    s, st = torch.zeros(B, D, dtype=torch.float64, device="cuda"), []
    for t in range(L):
        s = a[:, t] * s + u[:, t]
        st.append(s)
    yy = a3 * torch.stack(st, 1) + leaf["dsk"] * v
    out = norm(yy @ leaf["Wout"] + hh, leaf["w2"])
    out.backward(dout.double())

    def rel(got, want):
        return float((got.double() - want).norm() / want.norm())
    tol = 5 * 2.0 ** -8
    assert rel(n2, out.detach()) <= tol and rel(S, s.detach()) <= tol
    for got, k in ((g1.dresidual, "res"), (g1.dx, "x"), (g1.dweight, "w1"), (g2.dweight, "w2"), (gr.dlog_rate, "lr"),
                   (gr.dDskip, "dsk")):
        assert rel(got, leaf[k].grad) <= tol, k
    # the same layer one token at a time
    state = torch.zeros(B, D, **dev)
    for t in range(L):
        ht = torch.empty(B, D, **dev)
        pt = hy.rms_norm(x[:, t].contiguous(), w1, residual=res[:, t].contiguous(), residual_out=ht) @ Win
        yt = hy.gated_recurrence_decode(*(pt[:, i * D:(i + 1) * D] for i in range(4)), lr, dsk, state)
        nt = hy.rms_norm(yt @ Wout, w2, residual=ht)
        assert rel(nt, out[:, t].detach()) <= 2 * tol
    assert rel(state, s.detach()) <= tol
