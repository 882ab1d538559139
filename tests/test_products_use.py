"""The 8-bit products and the feed-forward block as programs use them: a whole
block of the model, captured graphs, other streams, several threads, workspaces
that serve more than one shape, tensors past 2^31 elements."""
import threading

import numpy as np
import pytest

from oracle import norm as onorm
from oracle import products as op

pytestmark = pytest.mark.gpu


def normal(*shape, seed, scale=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(torch.bfloat16).cuda()


def f64(t):
    return t.double().cpu().numpy()


def rel(got, ref):
    return float(np.linalg.norm(f64(got).ravel() - ref.ravel()) / np.linalg.norm(ref.ravel()))


@pytest.mark.parametrize("B,L", [(1, 1), (3, 1), (1, 300), (2, 129)])
def test_a_block(B, L):
    """norm -> in_proj -> modal convolution -> out_proj -> norm -> feed-forward -> down projection, all
    projections in e4m3, against the same in fp64 from the same codes at each step."""
    import torch
    import hyena_long_convolution_b200 as hy
    import oracle
    D, F, N, eps = 256, 704, 8, 1e-6
    M = B * L
    r = np.random.default_rng(L)
    weights = {k: normal(n, d, seed=i, scale=d ** -0.5)
               for i, (k, n, d) in enumerate((("in", 3 * D, D), ("out", D, D), ("gate", F, D), ("up", F, D), ("down", D, F)))}
    W = {k: hy.fp8_quantize(w, block=128) for k, w in weights.items()}
    V = {k: op.values(f64(q), f64(s), 128) for k, (q, s) in W.items()}
    wn = torch.ones(D, device="cuda")
    poles = torch.from_numpy(-np.exp(r.uniform(-6.9, 0.0, (D, N)))).float().cuda()
    res = torch.from_numpy(r.standard_normal((D, N)) / N).float().cuda()
    h = normal(B, L, D, seed=9)
    x = normal(B, L, D, seed=10)

    ho = torch.empty_like(h)
    q, s = hy.rms_norm_fp8(x, wn, eps, residual=h, residual_out=ho, group=128)
    z = hy.fp8_matmul(q, s, *W["in"])
    assert z.shape == (B, L, 3 * D)
    ref = op.values(f64(q).reshape(M, D), f64(s), 1) @ V["in"].T
    assert rel(z, ref) < 2.5e-3
    y = hy.modal_long_conv(z[..., :D], z[..., D:2 * D], z[..., 2 * D:], poles, res)
    yq, ys = hy.fp8_quantize(y)
    o = hy.fp8_matmul(yq, ys, *W["out"])
    assert rel(o, op.values(f64(yq).reshape(M, D), f64(ys), 1) @ V["out"].T) < 2.5e-3
    q2, s2 = hy.rms_norm_fp8(o, wn, eps, residual=ho, residual_out=ho)  # one scale a row
    fq, fs = hy.gated_ffn_fp8(q2, s2, *W["gate"], *W["up"], "gelu", fp8_out=True)
    ref = op.gated(op.values(f64(q2).reshape(M, D), f64(s2), 1), V["gate"], V["up"], "gelu")[0]
    got = op.values(f64(fq.float()).reshape(M, F), f64(fs), 1)
    assert np.linalg.norm(got - ref) < 2.0 ** -4 * np.linalg.norm(ref)
    d = hy.fp8_matmul(fq, fs, *W["down"])
    assert d.shape == (B, L, D) and rel(d, got @ V["down"].T) < 2.5e-3
    # and near the block in bf16 weights, all 8-bit roundings included
    n = onorm.forward(f64(ho).reshape(M, D), np.ones(D), eps)
    full = op.gated(n, f64(weights["gate"]), f64(weights["up"]), "gelu")[0] @ f64(weights["down"]).T
    assert rel(d, full) < 0.15


def test_training_step_and_checkpoint():
    """Forward keeping its products, gradient; a second forward (recomputed) gives the same bits."""
    import torch
    import hyena_long_convolution_b200 as hy
    x, wg, wu = normal(2, 150, 264, seed=0), normal(520, 264, seed=1, scale=264 ** -0.5), normal(520, 264, seed=2, scale=264 ** -0.5)
    dy = normal(2, 150, 520, seed=3)
    out = []
    for _ in range(2):
        g = torch.empty(2, 150, 520, device="cuda")
        u = torch.empty_like(g)
        y = hy.gated_ffn(x, wg, wu, "silu", gate_out=g, up_out=u)
        out.append((y, g, u, *hy.gated_ffn_backward(dy, x, wg, wu, g, u, "silu")))
    for a, b in zip(*out):
        assert torch.equal(a, b)
    X, DY = f64(x).reshape(300, 264), f64(dy).reshape(300, 520)
    _, rg, ru, _, _ = op.gated(X, f64(wg), f64(wu), "silu")
    for got, ref in zip(out[0][3:], op.gated_backward(DY, X, f64(wg), f64(wu), rg, ru, "silu")[:3]):
        assert rel(got, ref) < 5e-3
    # against torch's own differentiation of the formula, in fp64
    p = [t.double().requires_grad_() for t in (x, wg, wu)]
    (torch.nn.functional.silu(p[0] @ p[1].T) * (p[0] @ p[2].T) * dy.double()).sum().backward()
    for got, t in zip(out[0][3:], p):
        assert rel(got, f64(t.grad)) < 5e-3


def cases():
    import torch
    import hyena_long_convolution_b200 as hy
    wg, wu = (normal(1000, 528, seed=s, scale=528 ** -0.5) for s in (1, 2))
    qg, qu = (hy.fp8_quantize(w, block=128) for w in (wg, wu))
    for M in (1, 40, 150, 700):
        x = normal(M, 528, seed=M)
        q, s = hy.fp8_quantize(x)
        dy = normal(M, 1000, seed=M + 1)
        g, u = normal(M, 1000, seed=M + 2).float(), normal(M, 1000, seed=M + 3).float()
        yield lambda ws, x=x: hy.fp8_quantize(x)
        yield lambda ws, q=q, s=s: hy.fp8_matmul(q, s, *qg, workspace=ws)
        yield lambda ws, x=x: hy.gated_ffn(x, wg, wu, "gelu", workspace=ws)
        yield lambda ws, q=q, s=s: hy.gated_ffn_fp8(q, s, qg[0][:992], qg[1], qu[0][:992], qu[1], fp8_out=True, workspace=ws)
        yield lambda ws, dy=dy, x=x, g=g, u=u: hy.gated_ffn_backward(dy, x, wg, wu, g, u, workspace=ws)
    q, s = hy.fp8_quantize(normal(100, 4400, seed=5))
    w = hy.fp8_quantize(normal(9608, 4400, seed=6), block=128)  # 38 tiles of one CTA, three to each
    yield lambda ws: hy.fp8_matmul(q, s, *w, workspace=ws)


def same(a, b):
    import torch
    a, b = ([t] if isinstance(t, torch.Tensor) else list(t) for t in (a, b))
    return len(a) == len(b) and all(torch.equal(x.float(), y.float()) for x, y in zip(a, b))


def big_workspace():
    import hyena_long_convolution_b200 as hy
    return hy.FfnWorkspace(700, 528, 1000, backward=True)


def test_one_workspace_for_all():
    """Made for the most rows, it serves fewer, other entry points and the calls without one agree."""
    ws = big_workspace()
    for call in cases():
        first = call(None)
        assert same(call(ws), first) and same(call(ws), first)
    import hyena_long_convolution_b200 as hy
    hy.workspace_check(ws)


def test_graphs():
    import torch
    ws = [big_workspace() for _ in range(2)]
    for call in cases():
        want = call(None)
        graphs = []
        for w in ws:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                out = call(w)
            graphs.append((g, out))
        for _ in range(2):
            for g, out in graphs:
                for t in ([out] if isinstance(out, torch.Tensor) else out):
                    t.view(torch.uint8).zero_()
                g.replay()
                torch.cuda.synchronize()
                assert same(out, want)


def test_calls_in_a_row_see_each_other():
    """Each kernel starts before the one ahead ends: its reads must still come after."""
    import torch
    import hyena_long_convolution_b200 as hy
    w = torch.eye(256, device="cuda", dtype=torch.bfloat16)
    wq, sw = hy.fp8_quantize(w, block=128)
    for M in (2, 300):
        x = normal(M, 256, seed=M)
        want = x
        buf = [torch.empty_like(x) for _ in range(2)]
        q = torch.empty(M, 256, dtype=torch.float8_e4m3fn, device="cuda")
        s = torch.empty(M, 2, device="cuda")
        ws = hy.MatmulWorkspace(M, 256, 256)
        for i in range(30):  # the values are codes' own after the first turn, and stay
            hy.fp8_quantize(x if i == 0 else buf[(i + 1) % 2], q=q, scales=s)
            hy.fp8_matmul(q, s, wq, sw, y=buf[i % 2], workspace=ws)
        first = hy.fp8_matmul(*hy.fp8_quantize(want), wq, sw)
        assert rel(buf[1], f64(first)) < 2.0 ** -7 * 30
        x.zero_()
        hy.fp8_quantize(x, q=q, scales=s)
        x.fill_(1.0)  # after the quantiser has read it
        assert not hy.fp8_matmul(q, s, wq, sw).any()


@pytest.mark.parametrize("M", [128, 1024])
def test_before_a_kernel_that_reads_early(M):
    """The prepared modal convolution asks for its input rows before it waits for the kernel ahead of it."""
    import torch
    import hyena_long_convolution_b200 as hy
    D, N = 512, 8
    g = torch.Generator().manual_seed(0)
    poles = (-torch.exp(torch.rand(D, N, generator=g) * 6.9 - 6.9)).cuda()
    res = (torch.randn(D, N, generator=g) / N).cuda()
    ws = hy.ModalWorkspace(1, D, N)
    hy.modal_prepare(poles, res, None, ws)
    w, sw = hy.fp8_quantize(normal(3 * D, 4096, seed=1, scale=1 / 64), block=128)
    wide = hy.MatmulWorkspace(M, 3 * D, 4096)
    z = torch.empty(1, M, 3 * D, dtype=torch.bfloat16, device="cuda")
    xs = [z[..., i * D:(i + 1) * D] for i in range(3)]
    for seed in range(10):
        q, s = hy.fp8_quantize(normal(1, M, 4096, seed=seed))
        z.fill_(float("nan"))
        torch.cuda.synchronize()
        hy.fp8_matmul(q, s, w, sw, y=z, workspace=wide)
        y = hy.modal_long_conv_prepared(*xs, N, ws)
        torch.cuda.synchronize()
        assert torch.equal(y, hy.modal_long_conv_prepared(*xs, N, ws)), seed


@pytest.mark.parametrize("M,D,F", [(300, 1032, 1000), (1000, 264, 4104), (40, 2056, 520), (4000, 136, 264),
                                   (2000, 1032, 520), (4000, 2056, 264), (1, 4096, 4096)])
def test_what_follows_a_gradient_sees_all_of_it(M, D, F):
    """dW is worked out beside dx: the next kernel, of either kind, comes after both."""
    import torch
    import hyena_long_convolution_b200 as hy
    x, wg, wu = normal(M, D, seed=1), normal(F, D, seed=2, scale=D ** -0.5), normal(F, D, seed=3, scale=D ** -0.5)
    dy, g, u = normal(M, F, seed=4), normal(M, F, seed=5), normal(M, F, seed=6)
    ws = hy.FfnWorkspace(M, D, F, backward=True)
    want = hy.gated_ffn_backward(dy, x, wg, wu, g, u, workspace=ws)
    wq = [hy.fp8_quantize(t)[0].float() for t in want]
    out = [torch.empty_like(t) for t in want]
    for _ in range(10):
        for t in out:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        hy.gated_ffn_backward(dy, x, wg, wu, g, u, dx=out[0], dgate_weight=out[1], dup_weight=out[2], workspace=ws)
        copies = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(copies, want))
        hy.gated_ffn_backward(dy, x, wg, wu, g, u, dx=out[0], dgate_weight=out[1], dup_weight=out[2], workspace=ws)
        codes = [hy.fp8_quantize(t)[0] for t in out]
        assert all(torch.equal(a.float(), b) for a, b in zip(codes, wq))


def test_other_streams():
    import torch
    main = [call(None) for call in cases()]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        ws = big_workspace()
        side = [call(ws) for call in cases()]
    st.synchronize()
    assert all(same(a, b) for a, b in zip(main, side))
    import hyena_long_convolution_b200 as hy
    x = normal(3, 64, seed=0)
    w = normal(128, 64, seed=1)
    want = hy.gated_ffn(x, w, w)
    torch.cuda.synchronize()
    for s in (st, st.cuda_stream):
        y = hy.gated_ffn(x, w, w, stream=s)
        st.synchronize()
        assert torch.equal(y, want)


def test_threads():
    import torch
    want = [call(None) for call in cases()]
    torch.cuda.synchronize()
    bad = []

    def work():
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                ws = big_workspace()
                for _ in range(3):
                    got = [call(ws) for call in cases()]
                    st.synchronize()
                    if not all(same(a, b) for a, b in zip(got, want)):
                        bad.append("differs")
        except Exception as e:  # noqa: BLE001
            bad.append(repr(e))

    ts = [threading.Thread(target=work) for _ in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad


def test_workspace_too_small():
    import hyena_long_convolution_b200 as hy
    q, s = hy.fp8_quantize(normal(200, 128, seed=0))
    w, sw = hy.fp8_quantize(normal(128, 128, seed=1), block=128)
    with pytest.raises(hy.HyenaError) as e:
        hy.fp8_matmul(q, s, w, sw, workspace=hy.MatmulWorkspace(1, 128, 128))
    assert e.value.status == 6
    x, g = normal(200, 128, seed=2), normal(200, 128, seed=3)
    with pytest.raises(hy.HyenaError):
        hy.gated_ffn_backward(x, x, x[:128], x[:128], g, g, workspace=hy.FfnWorkspace(200, 128, 128))


@pytest.mark.slow
def test_past_2_to_31_elements():
    import torch
    import hyena_long_convolution_b200 as hy
    M, D, F = 270080, 64, 8192  # 2.2e9 outputs
    tail = slice(M - 256, M)
    x = torch.randn(M, D, device="cuda").to(torch.bfloat16)
    wg, wu = normal(F, D, seed=1, scale=D ** -0.5), normal(F, D, seed=2, scale=D ** -0.5)
    y = hy.gated_ffn(x, wg, wu)
    few = hy.gated_ffn(x[tail], wg, wu)
    assert torch.equal(y[tail], few) and torch.equal(y[:256], hy.gated_ffn(x[:256], wg, wu))
    q, s = hy.fp8_quantize(y)
    q2, s2 = hy.fp8_quantize(few)
    assert torch.equal(q[tail].float(), q2.float()) and torch.equal(s[tail], s2)
    w, sw = hy.fp8_quantize(normal(D, F, seed=3, scale=F ** -0.5), block=128)
    z, z2 = hy.fp8_matmul(q, s, w, sw), hy.fp8_matmul(q2, s2, w, sw)
    assert rel(z[tail], f64(z2)) < 4e-3
    del q, s, z
    g = y.float()[:, :0]  # keep y as both products: 2.2e9 values each
    del g
    d = hy.gated_ffn_backward(y, x, wg, wu, y, y, "identity")
    d2 = hy.gated_ffn_backward(few, x[tail], wg, wu, few, few, "identity")
    assert rel(d.dx[tail], f64(d2.dx)) < 4e-3
    ref = torch.zeros(128, D, dtype=torch.float64, device="cuda")
    for i in range(0, M, 16384):
        c = y[i:i + 16384, -128:].double()
        ref += (c * c).T @ x[i:i + 16384].double()
    assert rel(d.dgate_weight[-128:], f64(ref)) < 5e-3
