"""The 8-bit products, their quantiser and the gated feed-forward block against
their fp64 oracle, with tolerances that follow from the arithmetic.

With n = 2^-24 (half a step of fp32; 2 n for an addition that cuts off instead of
rounding, as a tensor core may): a sum over K products in fp32 is off by at most
2 n (K + 4) of the sum of its terms' absolute values; of codes, over each 128
channels and then over the groups, 2 n (128 + K / 128 + 8).  y = act(g) u takes
g's error by at most 1.2 |u|, u's by |act(g)|, and 16 n of |y| + |u| by itself.
The gradient's dg and du are rounded to bf16 (2^-8 of each) before their
products; their own arithmetic is off by at most 32 n (1 + |g|) of |dy u| and
|dy|.  Outputs add half a step of their type: bf16 2^-8, e4m3 2^-4 of the value
or 2^-10 among its subnormals.  These bounds add absolute values; over a whole
tensor of independent roundings the 2-norm of the error is at most 5e-3 of the
result's (one bf16 rounding: 2.3e-3; three: 4.0e-3).
"""
import numpy as np
import pytest

from oracle import products as op

pytestmark = pytest.mark.gpu

N = 2.0 ** -24
ACTS = ["silu", "gelu", "gelu_tanh", "identity"]


def f64(t):
    return t.double().cpu().numpy()


def near(got, ref, tol, what, half=0.0, rel=None):
    got = f64(got).reshape(ref.shape)
    assert np.isfinite(got).all(), what
    over = np.abs(got - ref) - (tol + half * np.abs(ref) + 1e-30)
    assert over.max() <= 0, f"{what}: over by {over.max():.3e} at {np.unravel_index(over.argmax(), ref.shape)}"
    if rel is not None and np.linalg.norm(ref) > 0:
        r = np.linalg.norm(got - ref) / np.linalg.norm(ref)
        assert r <= rel, f"{what}: {r:.3e} of the norm"


def inside(t, pad, fill):
    """t as a view of a larger buffer of `fill`: rows `pad` elements longer."""
    import torch
    big = torch.empty(t.shape[0] + 2, t.shape[1] + pad, dtype=torch.float32).fill_(fill).to(t.dtype).to(t.device)
    big[1:-1, :t.shape[1]] = t
    return big, big[1:-1, :t.shape[1]]


def codes(M, K, seed, block, per_row=False):
    """Random e4m3 codes of every size, and scales of a few binades."""
    import torch
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(M, K, generator=g) * 448 / 4).clamp(-448, 448).to(torch.float8_e4m3fn)
    rows = M if block == 1 else -(-M // block)
    s = torch.exp(torch.randn(rows, 1 if per_row else -(-K // 128), generator=g)) * K ** -0.25 / 100
    return q.cuda(), s.cuda()


def normal(*shape, seed, scale=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(torch.bfloat16).cuda()


# ------------------------------------------------------------------ quantiser

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("M,D", [(1, 8), (1, 4096), (3, 128), (5, 136), (127, 264), (128, 128), (129, 1032), (700, 520),
                                 (2, 16384)])
def test_quantize(M, D, block, dtype):
    import torch
    import hyena_long_convolution_b200 as hy
    g = torch.Generator().manual_seed(M + D)
    x = torch.randn(M, D, generator=g) * torch.exp(2 * torch.randn(M, 1, generator=g))
    x[M // 2] = 0
    x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    big, v = inside(x, 8, float("nan"))
    q, s = hy.fp8_quantize(v, block=block)
    ref = op.scales(f64(x), block)
    near(s, ref, 2 * N * ref, "scales")
    z = f64(x) / op.spread(ref, block, x.shape)
    near(q.float(), z, 8 * N * np.abs(z) + 2.0 ** -10, "q", 2.0 ** -4)
    # the codes are those of the fp32 quotient
    each = s.repeat_interleave(block, 0)[:M].repeat_interleave(128, 1)[:, :D]
    assert torch.equal(q.float(), (x.float() / each).to(torch.float8_e4m3fn).float())


def test_quantize_given_outputs_and_odd_values():
    import torch
    import hyena_long_convolution_b200 as hy
    x = torch.randn(4, 256, device="cuda")
    x[0, 3], x[1, 130], x[2] = float("inf"), float("nan"), 1e-38
    big, q = inside(torch.zeros(4, 256, device="cuda").to(torch.float8_e4m3fn), 16, 3.0)
    s = torch.empty(4, 2, device="cuda")
    got = hy.fp8_quantize(x, q=q, scales=s)
    assert got[0] is q and got[1] is s
    assert torch.isinf(s[0, 0]) and torch.isnan(s[1, 1]) and torch.isfinite(s[[0, 1], [1, 0]]).all()
    assert torch.isnan(q[0, 3].float()) and (q[0, :3].float() == 0).all() and torch.isnan(q[1, 128:].float()).all()
    assert (s[2] == 2.0 ** -100 / 448).all()
    out = big.float()
    out[1:-1, :256] = 3.0
    assert (out == 3.0).all()


# ---------------------------------------------------------------- 8-bit product

def check_matmul(M, Nn, K, per_row, dtype, seed=0):
    import torch
    import hyena_long_convolution_b200 as hy
    q, s = codes(M, K, seed + 1, 1, per_row)
    w, sw = codes(Nn, K, seed + 2, 128)
    Kp = -(-K // 16) * 16 - K
    _, qv = inside(q, Kp + 16, float("nan"))
    _, wv = inside(w, Kp, float("nan"))
    big, y = inside(torch.zeros(M, Nn, dtype=dtype, device="cuda"), 8, 7.0)
    hy.fp8_matmul(qv, s, wv, sw, y=y)
    x, wt = op.values(f64(q), f64(s), 1), op.values(f64(w), f64(sw), 128)
    tol = 2 * N * (128 + K / 128 + 8) * (np.abs(x) @ np.abs(wt).T)
    bf = dtype is torch.bfloat16
    near(y, x @ wt.T, tol, "y", 2.0 ** -8 if bf else 2 * N, rel=2.5e-3 if bf else None)
    out = big.float()
    out[1:-1, :Nn] = 7.0
    assert (out == 7.0).all(), "written outside y"


@pytest.mark.parametrize("M", [1, 2, 7, 16, 17, 33, 64, 65, 100, 128, 129, 200, 256, 300])
@pytest.mark.parametrize("Nn,K", [(8, 8), (128, 128), (136, 264), (264, 1040), (1032, 520), (520, 4096)])
def test_matmul(M, Nn, K):
    import torch
    check_matmul(M, Nn, K, M % 2 == 1, torch.float32, seed=M)


@pytest.mark.parametrize("M,Nn,K,per_row", [(1, 12288, 4096, True), (64, 4096, 11008, False), (999, 1032, 1040, False),
                                            (1024, 512, 640, True), (2049, 776, 256, False), (8, 40, 16384, False)])
def test_matmul_sizes(M, Nn, K, per_row):
    import torch
    check_matmul(M, Nn, K, per_row, torch.bfloat16)


# many rows by tiles of 256 x 256, whole or (few tiles, much k) in 2, 3 and 4 parts
@pytest.mark.parametrize("M,Nn,K", [(640, 2056, 264), (1300, 1160, 136), (257, 9608, 520), (2049, 1032, 1040),
                                    (300, 3328, 4400), (520, 1928, 4112), (300, 3336, 5200), (130, 4872, 8208)])
def test_matmul_many_rows(M, Nn, K):
    import torch
    check_matmul(M, Nn, K, False, torch.float32, seed=M)
    check_matmul(M, Nn, K, True, torch.bfloat16, seed=M)


@pytest.mark.parametrize("M,D,F,keep", [(300, 2056, 1664, "fp32"), (520, 136, 2696, "bf16"), (260, 4104, 1288, "bf16"),
                                        (700, 2184, 776, None)])
def test_ffn_many_rows(M, D, F, keep):
    import torch
    check_ffn(M, D, F, "gelu", {"fp32": torch.float32, "bf16": torch.bfloat16, None: None}[keep])


@pytest.mark.parametrize("M,D,F", [(300, 4400, 1936), (700, 272, 2064), (520, 5136, 1296), (1030, 528, 1040)])
def test_ffn_fp8_many_rows(M, D, F):
    check_ffn_fp8(M, D, F, "gelu_tanh", M % 3 == 1)


# tiles of 128 x 256, whole ones in one wave and in more, and in 2 and 3 parts; either side of the
# rows and columns where the kernels change
@pytest.mark.parametrize("M,Nn,K", [(33, 19080, 136), (64, 18944, 264), (64, 38152, 136), (100, 9608, 4400),
                                    (65, 14344, 4400), (128, 9480, 520), (300, 11008, 264), (390, 9608, 264),
                                    (1290, 8200, 136)])
def test_matmul_tiles_of_one_cta(M, Nn, K):
    import torch
    check_matmul(M, Nn, K, False, torch.float32, seed=M)
    check_matmul(M, Nn, K, True, torch.bfloat16, seed=M)


@pytest.mark.parametrize("M,D,F,keep", [(100, 264, 9608, "bf16"), (128, 136, 19080, None), (66, 72, 9480, "fp32"),
                                        (300, 136, 4872, "fp32"), (290, 264, 10248, "bf16"), (1200, 72, 4104, None)])
def test_ffn_tiles_of_one_cta(M, D, F, keep):
    import torch
    check_ffn(M, D, F, "silu", {"fp32": torch.float32, "bf16": torch.bfloat16, None: None}[keep])


@pytest.mark.parametrize("M,D,F", [(33, 272, 9616), (64, 144, 9488), (40, 272, 19088), (100, 4400, 4880),
                                   (128, 4400, 9344), (300, 144, 4880), (1200, 144, 4112), (390, 272, 9616)])
def test_ffn_fp8_tiles_of_one_cta(M, D, F):
    check_ffn_fp8(M, D, F, "gelu", M % 3 == 1)


def test_matmul_is_exact_on_whole_numbers():
    """Products and sums that fp32 holds exactly: every order gives the same."""
    import torch
    import hyena_long_convolution_b200 as hy
    g = torch.Generator().manual_seed(0)
    for M, Nn, K in ((1, 264, 4096), (20, 1000, 4096), (150, 264, 2064), (300, 520, 1040), (300, 3328, 4400),
                     (640, 2568, 272)):
        x = torch.randint(-8, 9, (M, K), generator=g).float()
        w = torch.randint(-8, 9, (Nn, K), generator=g).float()
        s = 2.0 ** torch.randint(-3, 4, (M, -(-K // 128)), generator=g).float()
        sw = 2.0 ** torch.randint(-3, 4, (-(-Nn // 128), -(-K // 128)), generator=g).float()
        e = torch.float8_e4m3fn
        y = hy.fp8_matmul(x.to(e).cuda(), s.cuda(), w.to(e).cuda(), sw.cuda(), dtype=torch.float32)
        ref = op.values(x.double().numpy(), s.double().numpy(), 1) @ op.values(w.double().numpy(), sw.double().numpy(),
                                                                             128).T
        assert (f64(y) == ref).all(), (M, Nn, K)


def test_matmul_keeps_nan_and_inf_where_they_are():
    import torch
    import hyena_long_convolution_b200 as hy
    for M in (3, 40, 200, 300):
        q, s = codes(M, 272, 1, 1)
        w, sw = codes(264, 272, 2, 128)
        clean = hy.fp8_matmul(q[:, :256], s[:, :2].contiguous(), w[:, :256], sw[:, :2].contiguous())
        q[1, 5] = float("nan")
        w[130, 7] = float("nan")
        s[2, 1] = float("inf")
        y = hy.fp8_matmul(q[:, :256], s[:, :2].contiguous(), w[:, :256], sw[:, :2].contiguous())
        assert torch.isnan(y[1]).all() and torch.isnan(y[:, 130]).all() and not torch.isfinite(y[2]).any()
        rows = [i for i in range(M) if i not in (1, 2)]
        keep = torch.tensor([j != 130 for j in range(264)])
        assert torch.equal(y[rows][:, keep], clean[rows][:, keep])


# ------------------------------------------------------------ feed-forward block

def inputs(M, D, F, seed):
    x = normal(M, D, seed=seed)
    return x, normal(F, D, seed=seed + 1, scale=D ** -0.5), normal(F, D, seed=seed + 2, scale=D ** -0.5)


def check_ffn(M, D, F, act, keep, seed=0):
    import torch
    import hyena_long_convolution_b200 as hy
    x, wg, wu = inputs(M, D, F, seed)
    _, xv = inside(x, 16, float("nan"))
    _, gv = inside(wg, 8, float("nan"))
    _, uv = inside(wu, 8, float("nan"))
    big, yv = inside(torch.zeros(M, F, dtype=torch.bfloat16, device="cuda"), 8, 7.0)
    g = u = None
    if keep:
        gbig, g = inside(torch.zeros(M, F, dtype=keep, device="cuda"), 24, 7.0)
        ubig, u = inside(torch.zeros(M, F, dtype=keep, device="cuda"), 24, 7.0)
    hy.gated_ffn(xv, gv, uv, act, y=yv, gate_out=g, up_out=u)
    ref, rg, ru, ag, au = op.gated(f64(x), f64(wg), f64(wu), act)
    tg, tu = 2 * N * (D + 4) * ag, 2 * N * (D + 4) * au
    a = np.abs(op.act(act, rg)[0])
    near(yv, ref, 1.2 * np.abs(ru) * tg + a * tu + tg * tu + 16 * N * (np.abs(ref) + np.abs(ru)), "y", 2.0 ** -8,
         rel=2.5e-3)
    if keep:
        half = 2.0 ** -8 if keep is torch.bfloat16 else N
        near(g, rg, tg, "gate", half)
        near(u, ru, tu, "up", half)
        for b in (gbig, ubig):
            out = b.float()
            out[1:-1, :F] = 7.0
            assert (out == 7.0).all(), "written outside the kept products"
    out = big.float()
    out[1:-1, :F] = 7.0
    assert (out == 7.0).all(), "written outside y"


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,D,F", [(1, 8, 8), (3, 64, 136), (17, 72, 264), (64, 128, 128), (65, 264, 72), (130, 1032, 392),
                                   (200, 64, 1000), (300, 520, 264)])
def test_ffn(M, D, F, act):
    import torch
    check_ffn(M, D, F, act, [None, torch.bfloat16, torch.float32][M % 3])


@pytest.mark.parametrize("M,D,F,keep", [(1, 4096, 2752, None), (16, 4096, 1000, "fp32"), (33, 2056, 2760, "bf16"),
                                        (100, 1000, 4104, None), (1000, 1032, 2760, "fp32"), (2050, 264, 136, "bf16")])
def test_ffn_sizes(M, D, F, keep):
    import torch
    check_ffn(M, D, F, "silu", {"fp32": torch.float32, "bf16": torch.bfloat16, None: None}[keep])


def check_ffn_fp8(M, D, F, act, per_row, seed=0):
    import torch
    import hyena_long_convolution_b200 as hy
    q, s = codes(M, D, seed + 1, 1, per_row)
    wg, sg = codes(F, D, seed + 2, 128)
    wu, su = codes(F, D, seed + 3, 128)
    # products of about unit size
    x = op.values(f64(q), f64(s), 1)
    sg, su = (t * float(2.0 ** -np.round(np.log2(np.std(x @ op.values(f64(w), f64(t), 128).T) + 1e-30)))
              for w, t in ((wg, sg), (wu, su)))
    _, qv = inside(q, 16, float("nan"))
    args = (qv, s, wg, sg.contiguous(), wu, su.contiguous(), act)
    y = hy.gated_ffn_fp8(*args)
    ref, rg, ru, ag, au = op.gated(x, op.values(f64(wg), f64(sg), 128), op.values(f64(wu), f64(su), 128), act)
    n = 2 * N * (128 + D / 128 + 8)
    tg, tu = n * ag, n * au
    tol = 1.2 * np.abs(ru) * tg + np.abs(op.act(act, rg)[0]) * tu + tg * tu + 16 * N * (np.abs(ref) + np.abs(ru))
    near(y, ref, tol, "y", 2.0 ** -8, rel=2.5e-3)
    if F % 16:
        return
    big, qo = inside(torch.zeros(M, F, device="cuda").to(torch.float8_e4m3fn), 16, 3.0)
    _, so = hy.gated_ffn_fp8(*args, fp8_out=True, q=qo)
    rs = op.scales(ref, 1)
    groups = [slice(i, i + 128) for i in range(0, F, 128)]
    ts = np.stack([tol[:, c].max(1) for c in groups], 1) / 448 + 4 * N * rs
    near(so, rs, ts, "scales")
    each, te = op.spread(rs, 1, ref.shape) if len(groups) > 1 else rs, \
        op.spread(ts, 1, ref.shape) if len(groups) > 1 else ts
    z = ref / each
    near(qo.float(), z, (1 + 2.0 ** -4) * (tol / each + np.abs(z) * te / each * 1.1) + 2.0 ** -10, "q", 2.0 ** -4)
    out = big.float()
    out[1:-1, :F] = 3.0
    assert (out == 3.0).all(), "written outside q"


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,D,F", [(1, 16, 16), (3, 64, 136), (17, 272, 256), (64, 128, 128), (65, 1040, 80),
                                   (130, 528, 400), (200, 64, 1008), (300, 528, 272)])
def test_ffn_fp8(M, D, F, act):
    check_ffn_fp8(M, D, F, act, M % 2 == 1)


@pytest.mark.parametrize("M,D,F", [(1, 4096, 2752), (16, 4096, 1008), (33, 2064, 2768), (100, 1008, 4112),
                                   (1000, 1040, 2768)])
def test_ffn_fp8_sizes(M, D, F):
    check_ffn_fp8(M, D, F, "silu", False)


def check_backward(M, D, F, act, keep, seed=0):
    import torch
    import hyena_long_convolution_b200 as hy
    x, wg, wu = inputs(M, D, F, seed)
    g, u = normal(M, F, seed=seed + 3).to(keep), normal(M, F, seed=seed + 4).to(keep)
    dy = normal(M, F, seed=seed + 5)
    views = [inside(t, 8, float("nan"))[1] for t in (dy, x, wg, wu, g, u)]
    outs = [inside(torch.zeros(*s, dtype=torch.bfloat16, device="cuda"), 8, 7.0) for s in ((M, D), (F, D), (F, D))]
    hy.gated_ffn_backward(*views, act, dx=outs[0][1], dgate_weight=outs[1][1], dup_weight=outs[2][1])
    X, Wg, Wu, G, U, DY = (f64(t) for t in (x, wg, wu, g, u, dy))
    dx, dwg, dwu, dg, du = op.gated_backward(DY, X, Wg, Wu, G, U, act)
    eg = 2.0 ** -8 * np.abs(dg) + 33 * N * (1 + np.abs(G)) * np.abs(DY * U)
    eu = 2.0 ** -8 * np.abs(du) + 33 * N * (1 + np.abs(G)) * np.abs(DY)
    ag, au = np.abs(dg) + eg, np.abs(du) + eu
    tx = eg @ np.abs(Wg) + eu @ np.abs(Wu) + 2 * N * (2 * F + 4) * (ag @ np.abs(Wg) + au @ np.abs(Wu))
    near(outs[0][1], dx, tx, "dx", 2.0 ** -8, rel=5e-3)
    for (_, got), want, e, a in ((outs[1], dwg, eg, ag), (outs[2], dwu, eu, au)):
        near(got, want, e.T @ np.abs(X) + 2 * N * (M + 4) * (a.T @ np.abs(X)), "dw", 2.0 ** -8, rel=5e-3)
    for (big, v) in outs:
        v.fill_(7.0)
        assert (big.float() == 7.0).all(), "written outside a gradient"


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,D,F", [(1, 8, 8), (3, 64, 136), (17, 72, 264), (64, 128, 128), (65, 264, 72), (130, 1032, 392),
                                   (200, 64, 1000), (300, 520, 264)])
def test_backward(M, D, F, act):
    import torch
    check_backward(M, D, F, act, [torch.bfloat16, torch.float32][M % 2])


@pytest.mark.parametrize("M,D,F", [(1, 2048, 2760), (1000, 1032, 2760), (2050, 264, 136), (5, 4096, 264)])
def test_backward_sizes(M, D, F):
    import torch
    check_backward(M, D, F, "gelu", torch.float32)


# dx by the weights' columns: clusters of 8, 4, 2 and none, one and several tiles of rows; and
# either side of where it is not
@pytest.mark.parametrize("M,D,F", [(17, 264, 1096), (520, 264, 1032), (100, 2056, 1096), (128, 4104, 520),
                                   (300, 1000, 1096), (64, 5000, 264), (40, 9608, 72), (900, 1032, 264),
                                   (1000, 1032, 264), (129, 4232, 72), (129, 4104, 136)])
def test_backward_few_rows(M, D, F):
    import torch
    check_backward(M, D, F, "silu", torch.float32 if M % 2 else torch.bfloat16, seed=M)


def test_no_rows():
    import torch
    import hyena_long_convolution_b200 as hy
    x, wg, wu = inputs(1, 64, 128, 0)
    none = x[:0]
    assert hy.gated_ffn(none, wg, wu).shape == (0, 128)
    e = none[:, :0].new_empty(0, 128)
    dw = [torch.ones(128, 72, dtype=torch.bfloat16, device="cuda")[:, :64] for _ in range(2)]
    g = hy.gated_ffn_backward(e, none, wg, wu, e, e, dgate_weight=dw[0], dup_weight=dw[1])
    assert g.dx.shape == (0, 64) and not dw[0].any() and not dw[1].any()
    assert (dw[0]._base[:, 64:] == 1).all()
    q, s = hy.fp8_quantize(none)
    wq, sw = hy.fp8_quantize(wg, block=128)
    assert q.shape == (0, 64) and s.shape == (0, 1)
    assert hy.fp8_matmul(q, s, wq, sw).shape == (0, 128)
    q, s = hy.gated_ffn_fp8(q, s, wq, sw, wq, sw, fp8_out=True)
    assert q.shape == (0, 128) and s.shape == (0, 1)


def test_infinite_gates():
    """Where act(g) of an infinite g is finite or infinite, y is what the formula gives."""
    import torch
    import hyena_long_convolution_b200 as hy
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    x[0, 0], x[1, 0] = float("inf"), 1.0
    w = torch.zeros(128, 64, dtype=torch.bfloat16, device="cuda")
    w[:, 0] = 1.0
    for act in ACTS:
        y = hy.gated_ffn(x, w, w, act)
        assert (y[0] == float("inf")).all() and torch.isfinite(y[1]).all()
