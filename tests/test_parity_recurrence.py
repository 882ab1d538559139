"""The gated recurrence (forward, gradient, decode) against its fp64 oracle,
with tolerances that follow from the kernels' arithmetic.

With h = 2^-24 (half a step of fp32) and |gate| <= 8:
  * sigmoid: exp(-gate) as 2^t, t rounded (16 h relative at |gate| = 8), 2 units
    of ex2 (4 h), the sum and the reciprocal (3 h): 23 h, and l = rate sigmoid 24 h;
  * a: |l| a <= 1/e, so l's error moves a by at most 9 h; the polynomial, the
    exponent of the large branch and the final rounding 6 h more: 15 h absolute;
  * w = sqrt(1 - a^2): 1 - a is formed relative to itself (38 h), the root halves
    it, its own rounding 2 h: 22 h relative; u = w v: 23 h;
  * so one token adds at most 15 h |s| + 23 h |u| + h |s| to the error that it
    carries on with weight a, and a segment's or unit's decay (from the sum of
    its l) less than the tokens it covers: |s error| <= 40 L h S, with S the
    same sum over absolute values.  q, from the right, likewise.
  * products add their factors' errors; the square of w below costs 2 x 22 h,
    sigmoid (1 - sigmoid) 2 x 23 h, the sums over tokens (8 in a segment, 8
    segments, then double) 20 h.
bf16 outputs add half a step, 2^-8 of the value.
"""
import numpy as np
import pytest

from oracle import recurrence as orec

pytestmark = pytest.mark.gpu

H = 2.0 ** -24
UNIT = 64


def make(B, L, D, seed, state=True, skip=True, resets=None, dtype=np.float64):
    import torch
    g = torch.Generator().manual_seed(seed)
    d = {k: torch.randn(B, L, D, generator=g).to(torch.bfloat16) for k in ("x1", "x2", "x3", "dy")}
    d["gate"] = (2.0 * torch.randn(B, L, D, generator=g)).clamp(-8, 8).to(torch.bfloat16)
    d["log_rate"] = -torch.exp(torch.rand(D, generator=g) * 9.0 - 6.9)  # 1e-3 .. 8
    d["Dskip"] = torch.randn(D, generator=g) if skip else None
    d["state_in"] = torch.randn(B, D, generator=g) if state else None
    d["dstate_out"] = torch.randn(B, D, generator=g) if state else None
    r = None
    if resets is not None:
        r = torch.zeros(B, L, dtype=torch.bool)
        if resets == "all":
            r[:] = True
        elif resets == "first":
            r[:, 0] = True
        elif resets == "last":
            r[:, -1] = True
        else:
            r = torch.rand(B, L, generator=g) < resets
            r[0] = False  # one row without any
    d["reset"] = r
    return d


def cuda(d):
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def f64(d):
    return {k: None if v is None else (v.numpy() if v.dtype.is_floating_point is False else v.double().numpy())
            for k, v in d.items()}


FWD = ("x1", "x2", "x3", "gate", "log_rate", "Dskip")


def run_forward(hy, d, normalize, **kw):
    import torch
    B, L, D = d["x1"].shape
    out = torch.empty(B, D, device="cuda")
    units = hy.recurrence_unit_states(B, L, D)
    y = hy.gated_recurrence(*(d[k] for k in FWD), reset=d["reset"], normalize=normalize, state_in=d["state_in"],
                            state_out=out, unit_states=units, **kw)
    return y, out, units


def run_backward(hy, d, units, normalize, **kw):
    return hy.gated_recurrence_backward(d["dy"], *(d[k] for k in FWD), units, reset=d["reset"], normalize=normalize,
                                        dstate_out=d["dstate_out"], **kw)


def bits(t):
    import torch
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32).cpu().numpy()


def same(a, b):
    return np.array_equal(bits(a), bits(b))


def near(got, ref, tol, what, half=0.0):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    over = np.abs(got - ref) - (tol + half * np.abs(ref) + 1e-30)
    assert over.max() <= 0, f"{what}: off by {np.abs(got - ref).flat[over.argmax()]:.3e}, over by {over.max():.3e}"


def check(d, normalize, y, state, units, grads):
    n = f64(d)
    L = n["x1"].shape[1]
    kw = dict(reset=n["reset"], normalize=normalize, state_in=n["state_in"])
    f = orec.forward(*(n[k] for k in FWD), **kw)
    T = 40 * L * H
    half = 2.0 ** -8
    v = np.abs(n["x1"] * n["x2"])
    ds = 0.0 if n["Dskip"] is None else np.abs(n["Dskip"])
    # y = x3 s + Dskip v: two more roundings of the parts
    near(y, f.y, (T + 2 * H) * np.abs(n["x3"]) * f.scale + 2 * H * ds * v, "y", half)
    near(state, f.state_out, T * f.scale[:, -1], "state_out")
    starts = np.concatenate([np.zeros_like(f.states[:, :1]) if n["state_in"] is None else n["state_in"][:, None],
                             f.states[:, UNIT - 1:-1:UNIT]], 1)
    scale = np.concatenate([np.abs(starts[:, :1]), f.scale[:, UNIT - 1:-1:UNIT]], 1)
    near(units, starts, T * scale, "unit_states")
    if grads is None:
        return
    b = orec.backward(n["dy"], *(n[k] for k in FWD), dstate_out=n["dstate_out"], **kw)
    T2 = 2 * T + 200 * H  # two carried factors and the gates' derivatives
    for k in ("dx1", "dx2", "dx3", "dgate"):
        near(getattr(grads, k), getattr(b, k), T2 * b.scales[k], k, half)
    near(grads.dlog_rate, b.dlog_rate, T2 * b.scales["dlog_rate"], "dlog_rate")
    near(grads.dstate_in, b.dstate_in, (T + 16 * H) * b.scales["dstate_in"], "dstate_in")
    if n["Dskip"] is None:
        assert grads.dDskip is None
    else:
        near(grads.dDskip, b.dDskip, 20 * H * b.scales["dDskip"], "dDskip")


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("B,L,D,state,skip,resets", [
    (1, 1, 8, True, True, None), (1, 1, 8, False, False, "all"), (2, 2, 8, True, True, None),
    (1, 7, 64, False, True, 0.3), (3, 8, 72, True, False, "first"), (1, 9, 64, True, True, "last"),
    (2, 63, 200, True, True, None), (1, 64, 64, True, True, "first"), (2, 65, 136, False, False, 0.05),
    (1, 128, 64, True, True, "all"), (2, 130, 72, True, True, 0.02), (3, 300, 264, True, True, None),
    (1, 1000, 64, False, True, 0.003), (5, 257, 8, True, False, 0.01),
])
def test_matches_oracle(B, L, D, state, skip, resets, normalize):
    import hyena_long_convolution_b200 as hy
    d = make(B, L, D, seed=B + 10 * L + D, state=state, skip=skip, resets=resets)
    c = cuda(d)
    y, s, units = run_forward(hy, c, normalize)
    g = run_backward(hy, c, units, normalize)
    check(d, normalize, y, s, units, g)


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("resets", [None, 0.02])
def test_chunks_of_whole_units_are_the_single_pass(normalize, resets):
    import torch
    import hyena_long_convolution_b200 as hy
    B, L, D = 2, 5 * UNIT + 17, 72
    c = cuda(make(B, L, D, seed=3, resets=resets))
    y, s, units = run_forward(hy, c, normalize)
    g = run_backward(hy, c, units, normalize)
    cuts = [0, UNIT, 4 * UNIT, L]
    seq = ("x1", "x2", "x3", "gate", "dy", "reset")
    parts = [{k: v[:, a:b].contiguous() if k in seq and v is not None else v for k, v in c.items()}
             for a, b in zip(cuts, cuts[1:])]
    S = c["state_in"].clone()
    states = []
    for p, a, b in zip(parts, cuts, cuts[1:]):
        u = hy.recurrence_unit_states(B, b - a, D)
        yc = hy.gated_recurrence(*(p[k] for k in FWD), reset=p["reset"], normalize=normalize, state_in=S,
                                 state_out=S, unit_states=u)
        states.append(u)
        assert same(yc, y[:, a:b])
    assert same(S, s) and same(torch.cat(states, 1), units)
    e = c["dstate_out"].clone()
    for p, u, a, b in list(zip(parts, states, cuts, cuts[1:]))[::-1]:
        gc = hy.gated_recurrence_backward(p["dy"], *(p[k] for k in FWD), u, reset=p["reset"], normalize=normalize,
                                          dstate_out=e, dstate_in=e)
        for k in ("dx1", "dx2", "dx3", "dgate"):
            assert same(getattr(gc, k), getattr(g, k)[:, a:b]), k
    assert same(e, g.dstate_in)


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("B,D", [(1, 8), (3, 200), (2, 4096), (70, 64)])
def test_decode_is_the_one_token_pass(B, D, normalize):
    import hyena_long_convolution_b200 as hy
    d = make(B, 1, D, seed=B + D, skip=D != 200)
    c = cuda(d)
    y, s, _ = run_forward(hy, c, normalize)
    S = c["state_in"].clone()
    yd = hy.gated_recurrence_decode(*(c[k] for k in FWD), S, normalize=normalize)
    assert same(yd, y) and same(S, s)
    S = c["state_in"].clone()
    yd = hy.gated_recurrence_decode(*(c[k][:, 0] if c[k] is not None and c[k].dim() == 3 else c[k] for k in FWD), S,
                                    normalize=normalize)
    assert same(yd, y[:, 0]) and same(S, s)


def test_prefill_then_decode_follows_the_oracle():
    import torch
    import hyena_long_convolution_b200 as hy
    B, L, T, D = 2, 100, 20, 72
    d = make(B, L + T, D, seed=21)
    c = cuda(d)
    S = torch.empty(B, D, device="cuda")
    head = {k: v[:, :L].contiguous() if k in ("x1", "x2", "x3", "gate") else v for k, v in c.items()}
    ys = [hy.gated_recurrence(*(head[k] for k in FWD), state_in=c["state_in"], state_out=S)]
    for t in range(L, L + T):
        ys.append(hy.gated_recurrence_decode(*(c[k][:, t:t + 1] for k in FWD[:4]), c["log_rate"], c["Dskip"], S))
    f = orec.forward(*(f64(d)[k] for k in FWD), state_in=f64(d)["state_in"])
    n = f64(d)
    T_ = 40 * (L + T) * H
    near(torch.cat(ys, 1), f.y, (T_ + 2 * H) * np.abs(n["x3"]) * f.scale
         + 2 * H * np.abs(n["Dskip"] * n["x1"] * n["x2"]), "y", 2.0 ** -8)
    near(S, f.state_out, T_ * f.scale[:, -1], "state")


def test_views_of_one_projection_and_padded_outputs():
    """x1, x2, x3, gate as views of one [B, L, 4D] buffer; y and the gradients
    as views whose padding stays as it was."""
    import torch
    import hyena_long_convolution_b200 as hy
    B, L, D, pad = 2, 150, 72, 8
    d = cuda(make(B, L, D, seed=31))
    y, s, units = run_forward(hy, d, True)
    g = run_backward(hy, d, units, True)
    proj = torch.cat([d[k] for k in ("x1", "x2", "x3", "gate")], 2)
    v = dict(d, **{k: proj[:, :, i * D:(i + 1) * D] for i, k in enumerate(("x1", "x2", "x3", "gate"))})
    dyp = torch.full((B, L, D + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    dyp[..., :D] = d["dy"]
    v["dy"] = dyp[..., :D]
    yp = torch.full((B, L, D + pad), 3.0, dtype=torch.bfloat16, device="cuda")
    y2, s2, units2 = run_forward(hy, v, True, y=yp[..., :D])
    assert same(yp[..., :D], y) and same(s2, s) and same(units2, units)
    assert (yp[..., D:] == 3.0).all()
    gp = torch.full((B, L, 4 * D + pad), 5.0, dtype=torch.bfloat16, device="cuda")
    parts = [gp[:, :, i * D:(i + 1) * D] for i in range(4)]
    g2 = run_backward(hy, v, units2, True, dx1=parts[0], dx2=parts[1], dx3=parts[2], dgate=parts[3])
    for k, t in zip(("dx1", "dx2", "dx3", "dgate"), parts):
        assert same(t, getattr(g, k)), k
    assert same(g2.dlog_rate, g.dlog_rate) and same(g2.dDskip, g.dDskip) and same(g2.dstate_in, g.dstate_in)
    assert (gp[..., 4 * D:] == 5.0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("at", [0, 5, 63, 64, 100, 199])
def test_nothing_passes_a_reset(bad, at):
    """A token that is not finite spoils its own sequence and channel only, in
    both directions."""
    import torch
    import hyena_long_convolution_b200 as hy
    B, L, D = 1, 200, 64
    d = make(B, L, D, seed=41, resets="first")
    d["reset"][0, [10, 64, 90, 130]] = True
    clean = cuda(d)
    y0, s0, u0 = run_forward(hy, clean, True)
    g0 = run_backward(hy, clean, u0, True)
    spoilt = dict(clean, x1=clean["x1"].clone(), dy=clean["dy"].clone(), state_in=clean["state_in"].clone())
    spoilt["x1"][0, at, 3] = bad
    spoilt["dy"][0, at, 3] = bad
    spoilt["state_in"][0, 3] = bad  # cut at token 0
    y, s, u = run_forward(hy, spoilt, True)
    g = run_backward(hy, spoilt, u, True)
    starts = [0, 10, 64, 90, 130, L]
    lo = max(t for t in starts if t <= at)
    hi = min(t for t in starts if t > at)
    assert not np.isfinite(y[0, at:hi, 3].double().cpu().numpy()).any()
    keep = torch.ones(B, L, D, dtype=torch.bool, device="cuda")
    keep[0, lo:hi, 3] = False
    assert torch.equal(y[keep], y0[keep])
    for k in ("dx1", "dx2", "dx3", "dgate"):
        a, b = getattr(g, k), getattr(g0, k)
        assert torch.equal(a[keep], b[keep]), k
    ch = torch.arange(D, device="cuda") != 3
    assert torch.equal(g.dlog_rate[ch], g0.dlog_rate[ch])
    if hi < L:
        assert torch.equal(s, s0)
    assert torch.equal(g.dstate_in[:, ch], g0.dstate_in[:, ch])
    assert (g.dstate_in[0, 3] == 0).all()  # nothing passes the reset at token 0


def test_extreme_gates_and_rates():
    """Saturated gates, a rate of zero, rates that decay within a token."""
    import torch
    import hyena_long_convolution_b200 as hy
    B, L, D = 1, 70, 64
    d = make(B, L, D, seed=51)
    gates = torch.tensor([-3e38, -1e4, -200.0, -88.0, -60.0, 30.0, 100.0, 3e38], dtype=torch.bfloat16)
    d["gate"][0, :, :] = gates[torch.arange(L * D).view(L, D) % 8]
    d["log_rate"][::4] = 0.0
    d["log_rate"][1::4] = -1e4
    d["log_rate"][2::4] = -1e-30
    c = cuda(d)
    for normalize in (True, False):
        y, s, units = run_forward(hy, c, normalize)
        g = run_backward(hy, c, units, normalize)
        for t in (y, s, units, *(x for x in g)):
            assert torch.isfinite(t).all()
        n = f64(d)
        f = orec.forward(*(n[k] for k in FWD), normalize=normalize, state_in=n["state_in"])
        # |gate| > 8 loses digits of exp(-gate) where the sigmoid is below e^-8; 87 (2 h) of |l| each
        T = 40 * L * H + 200 * H
        near(s, f.state_out, T * f.scale[:, -1] + 1e-12, "state_out")
        near(y, f.y, T * np.abs(n["x3"]) * f.scale + 1e-12 + 2 * H * np.abs(n["Dskip"] * n["x1"] * n["x2"]), "y",
             2.0 ** -8)


def test_nan_gate_and_rate_propagate():
    import torch
    import hyena_long_convolution_b200 as hy
    c = cuda(make(1, 80, 64, seed=52))
    c["gate"][0, 40, 7] = float("nan")
    c["log_rate"][9] = float("nan")
    y, s, _ = run_forward(hy, c, True)
    assert torch.isnan(y[0, 40:, 7]).all() and torch.isfinite(y[0, :40, 7]).all()
    assert torch.isnan(y[0, :, 9]).all()
    ok = [i for i in range(64) if i not in (7, 9)]
    assert torch.isfinite(y[:, :, ok]).all() and torch.isfinite(s[:, ok]).all()


def test_empty_sequence():
    import torch
    import hyena_long_convolution_b200 as hy
    d = cuda(make(2, 0, 64, seed=61))
    y, s, units = run_forward(hy, d, True)
    assert y.shape == (2, 0, 64) and units.shape == (2, 0, 64) and same(s, d["state_in"])
    g = run_backward(hy, d, units, True)
    assert same(g.dstate_in, d["dstate_out"]) and (g.dlog_rate == 0).all() and (g.dDskip == 0).all()
    d["state_in"] = d["dstate_out"] = None
    _, s, units = run_forward(hy, d, True)
    assert (s == 0).all() and (run_backward(hy, d, units, True).dstate_in == 0).all()


def test_one_workspace_many_shapes_streams_and_graphs():
    """One workspace serves calls of any shape that fits; calls on another
    stream and in replayed graphs give the same bits."""
    import torch
    import hyena_long_convolution_b200 as hy
    ws = hy.RecurrenceWorkspace(2, 1000, 200)
    shapes = [(2, 1000, 200), (1, 70, 64), (2, 129, 200), (1, 1, 8), (1, 3000, 64)]
    ref = []
    for B, L, D in shapes:
        c = cuda(make(B, L, D, seed=L, resets=0.01))
        y, s, u = run_forward(hy, c, True)
        ref.append((c, y, s, u, run_backward(hy, c, u, True)))
    for _ in range(3):
        for c, y, s, u, g in ref:
            y2, s2, u2 = run_forward(hy, c, True, workspace=ws)
            g2 = run_backward(hy, c, u2, True, workspace=ws)
            assert same(y, y2) and same(s, s2) and same(u, u2)
            assert all(same(a, b) for a, b in zip(g, g2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c, y, s, u, g = ref[0]
    ws2 = hy.RecurrenceWorkspace(2, 1000, 200, stream=side)
    with torch.cuda.stream(side):
        y2, s2, u2 = run_forward(hy, c, True, workspace=ws2)
        g2 = run_backward(hy, c, u2, True, workspace=ws2)
    side.synchronize()
    assert same(y, y2) and all(same(a, b) for a, b in zip(g, g2))
    # the stream given instead of made current, as an object and as a handle; scratch of the call's own
    for st in (side, side.cuda_stream):
        y2, s2, u2 = run_forward(hy, c, True, stream=st)
        g2 = run_backward(hy, c, u2, True, stream=st)
        d2 = hy.gated_recurrence_decode(*(c[k][:, 0] for k in FWD[:4]), c["log_rate"], c["Dskip"],
                                        c["state_in"].clone(), stream=st)
        side.synchronize()
        assert same(y, y2) and all(same(a, b) for a, b in zip(g, g2)) and d2.shape == (2, 200)
    graphs, outs = [], []
    for c, *_ in (ref[0], ref[2]):  # two graphs, one workspace, replayed in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y2, s2, u2 = run_forward(hy, c, True, workspace=ws)
            g2 = run_backward(hy, c, u2, True, workspace=ws)
        graphs.append(graph)
        outs.append((y2, s2, u2, g2))
    for _ in range(3):
        for graph, out, (c, y, s, u, g) in zip(graphs, outs, (ref[0], ref[2])):
            for t in out[:3]:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert same(out[0], y) and same(out[1], s) and same(out[2], u)
            assert all(same(a, b) for a, b in zip(out[3], g))
    hy.workspace_check(ws)
    del graphs


def test_calls_at_once_from_several_threads_and_streams():
    """Launches that share the device, each with a workspace of its own and none
    with all of its CTAs resident, give the bits they give alone."""
    import threading

    import torch

    import hyena_long_convolution_b200 as hy
    cases = [cuda(make(2, 4000, 1032, seed=21)), cuda(make(1, 9000, 2048, seed=22)), cuda(make(1, 20000, 64, seed=23))]
    want = []
    for c in cases:
        y, s, u = run_forward(hy, c, True)
        want.append((y, s, u, run_backward(hy, c, u, True)))
    torch.cuda.synchronize()
    got, failed = [None] * 3, []

    def work(k):
        try:
            st = torch.cuda.Stream()
            B, L, D = cases[k]["x1"].shape
            with torch.cuda.stream(st):
                ws = hy.RecurrenceWorkspace(B, L, D)
                for _ in range(10):
                    y, s, u = run_forward(hy, cases[k], True, workspace=ws)
                    g = run_backward(hy, cases[k], u, True, workspace=ws)
                hy.workspace_check(ws)
            st.synchronize()
            got[k] = (y, s, u, g)
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for (y, s, u, g), (y2, s2, u2, g2) in zip(got, want):
        assert same(y, y2) and same(s, s2) and same(u, u2) and all(same(a, b) for a, b in zip(g, g2))


def test_launches_are_told_apart_past_32_bits():
    """The records' tags count launches in 64 bits: where the lower half goes
    round, zero-filled records and those of a launch with the same lower half are
    not taken for this launch's."""
    import torch

    import hyena_long_convolution_b200 as hy
    c, d = cuda(make(2, 1500, 136, seed=11)), cuda(make(2, 1500, 136, seed=12))
    want = run_forward(hy, d, True)
    grads = run_backward(hy, d, want[2], True)
    ws = hy.RecurrenceWorkspace(2, 1500, 136)
    launches = ws.buf[16:24].view(torch.int64)
    for before in (0, 2 ** 32 - 1, 2 ** 32, 2 ** 40):
        launches.fill_(before)
        assert all(same(x, y) for x, y in zip(run_forward(hy, d, True, workspace=ws), want))
        assert launches.item() == before + 1
        run_forward(hy, c, True, workspace=ws)
        assert all(same(x, y) for x, y in zip(run_backward(hy, d, want[2], True, workspace=ws), grads))
        hy.workspace_check(ws)


@pytest.mark.parametrize("B,L,D", [(1, 8192, 4096), (4, 2000, 1032), (1, 20000, 64)])
def test_long_sequences_against_a_64_bit_scan(B, L, D):
    """Lengths the numpy oracle is slow for: the same recurrence in torch's
    float64 on the device, the whole tensors compared.  A token adds at most
    16 h |s| + 23 h |u| of either sign (see above); carried on with weights
    a^k, the errors of M = 1 / (1 - a) <= L remembered tokens add in the root
    mean square to 16 h sqrt(M / 2) |s|, so the state is within (16 sqrt(L / 2)
    + 40) h of its norm, and a sum over two carried factors within twice that."""
    import torch
    import hyena_long_convolution_b200 as hy
    c = cuda(make(B, L, D, seed=L, resets=0.001))
    c["reset"][:] |= False
    y, s, units = run_forward(hy, c, True)
    x1, x2, x3, gate = (c[k].double() for k in ("x1", "x2", "x3", "gate"))
    l = c["log_rate"].double() * torch.sigmoid(gate)
    r = c["reset"][..., None]
    a = l.exp().masked_fill(r, 0.0)
    w = (-torch.expm1(2 * l)).sqrt().masked_fill(r, 1.0)
    u = w * x1 * x2
    st, S = torch.empty_like(u), c["state_in"].double()
    for t in range(L):
        S = torch.addcmul(u[:, t], a[:, t], S)
        st[:, t] = S
    ref = x3 * st + c["Dskip"].double() * x1 * x2

    def rel(got, want):
        return float((got.double() - want).norm() / want.norm())
    T = (16 * (L / 2) ** 0.5 + 40) * H
    assert rel(y, ref) <= 2.0 ** -8
    assert rel(s, S) <= T
    q, e = torch.empty_like(u), c["dstate_out"].double()
    rdy = x3 * c["dy"].double()
    for t in range(L - 1, -1, -1):
        q[:, t] = rdy[:, t] + e
        e = a[:, t] * q[:, t]
    g = run_backward(hy, c, units, True)
    prev = torch.cat([c["state_in"].double()[:, None], st[:, :-1]], 1)
    dl = a * q * (prev - a * x1 * x2 / w)
    sig = torch.sigmoid(gate)
    dv = w * q + c["Dskip"].double() * c["dy"].double()
    for k, want in (("dx1", dv * x2), ("dx2", dv * x1), ("dx3", c["dy"].double() * st),
                    ("dgate", dl * c["log_rate"].double() * sig * (1 - sig))):
        assert rel(getattr(g, k), want) <= 2.0 ** -8, k
    assert rel(g.dlog_rate, (dl * sig).sum((0, 1))) <= 2 * T
    assert rel(g.dDskip, (c["dy"].double() * x1 * x2).sum((0, 1))) <= 20 * H
    assert rel(g.dstate_in, e) <= T


@pytest.mark.slow
def test_offsets_past_32_bits():
    """A sequence of more than 2^31 elements: the tail of the single pass is
    the tail of the same sequence fed in two chunks (the inputs share memory)."""
    import torch
    import hyena_long_convolution_b200 as hy
    L, D, cut = 1048576 + 128 + 5, 2048, 524288
    x = torch.randn(1, L, D, dtype=torch.bfloat16, device="cuda")
    lr = -torch.exp(torch.rand(D, device="cuda") * 9.0 - 6.9)
    ws = hy.RecurrenceWorkspace(1, L, D)
    s, s2 = torch.empty(1, D, device="cuda"), torch.empty(1, D, device="cuda")
    y = hy.gated_recurrence(x, x, x, x, lr, state_out=s, workspace=ws)
    hy.workspace_check(ws)
    hy.gated_recurrence(*([x[:, :cut]] * 4), lr, state_out=s2, workspace=ws)
    y2 = hy.gated_recurrence(*([x[:, cut:]] * 4), lr, state_in=s2, state_out=s2, workspace=ws)
    assert same(s, s2) and torch.equal(y[:, cut:], y2)
