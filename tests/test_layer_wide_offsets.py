"""The recurrence's gradient and the norm over more than 2^31 elements, against
the same calls on parts of them; and resets given as bytes."""
import pytest

from .test_parity_recurrence import cuda, make, run_backward, run_forward, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [1, 255])
def test_resets_as_bytes(value):
    import torch
    import hyena_long_convolution_b200 as hy
    c = cuda(make(3, 300, 136, seed=9, resets=0.05))
    y, s, units = run_forward(hy, c, True)
    g = run_backward(hy, c, units, True)
    d = dict(c, reset=c["reset"].to(torch.uint8) * value)
    y2, s2, units2 = run_forward(hy, d, True)
    assert same(y2, y) and same(s2, s) and same(units2, units)
    assert all(same(a, b) for a, b in zip(run_backward(hy, d, units2, True), g))


@pytest.mark.slow
def test_recurrence_gradient():
    """The single pass against two chunks from the last to the first."""
    import torch
    import hyena_long_convolution_b200 as hy
    L, D, cut = 1048576 + 128 + 5, 2048, 524288
    x = torch.randn(1, L, D, dtype=torch.bfloat16, device="cuda")
    dy = torch.randn(1, L, D, dtype=torch.bfloat16, device="cuda")
    lr = -torch.exp(torch.rand(D, device="cuda") * 9.0 - 6.9)
    ws = hy.RecurrenceWorkspace(1, L, D)
    units = hy.recurrence_unit_states(1, L, D)
    hy.gated_recurrence(x, x, x, x, lr, unit_states=units, workspace=ws)
    g = hy.gated_recurrence_backward(dy, x, x, x, x, lr, None, units, workspace=ws)
    e, parts = None, []
    for a, b in ((cut, L), (0, cut)):
        u = units[:, a // 64:-(-b // 64)]
        xs = x[:, a:b]
        p = hy.gated_recurrence_backward(dy[:, a:b], xs, xs, xs, xs, lr, None, u, dstate_out=e, workspace=ws)
        for k in ("dx1", "dx2", "dx3", "dgate"):
            assert torch.equal(getattr(p, k), getattr(g, k)[:, a:b]), k
        e = p.dstate_in
        parts.append(p.dlog_rate)
    hy.workspace_check(ws)
    assert same(e, g.dstate_in)
    # the same units' parts, summed in double either way and rounded to fp32: half a step of each chunk's sum
    # and of the whole one's, which is no larger than both together
    both = parts[0].double() + parts[1].double()
    assert ((both - g.dlog_rate.double()).abs() <= 2 * 2.0 ** -24 * (parts[0].abs() + parts[1].abs()).double()).all()


@pytest.mark.slow
def test_norm():
    """The last rows against a call on them alone."""
    import torch
    import hyena_long_convolution_b200 as hy
    M, D, n = 2 ** 31 // 16384 + 1111, 16384, 1000
    x = torch.randn(M, D, dtype=torch.bfloat16, device="cuda")
    r = torch.randn(M, D, device="cuda")
    w = 1 + 0.1 * torch.randn(D, device="cuda")
    rstd = torch.empty(M, device="cuda")
    h = torch.empty_like(r)
    y = hy.rms_norm(x, w, residual=r, residual_out=h, rstd=rstd)
    h1, rstd1 = torch.empty_like(r[-n:]), torch.empty(n, device="cuda")
    assert torch.equal(hy.rms_norm(x[-n:], w, residual=r[-n:], residual_out=h1, rstd=rstd1), y[-n:])
    assert torch.equal(h1, h[-n:]) and torch.equal(rstd1, rstd[-n:])
    for group in (0, 128):
        q, s = hy.rms_norm_fp8(x, w, residual=r, group=group)
        q1, s1 = hy.rms_norm_fp8(x[-n:], w, residual=r[-n:], group=group)
        assert torch.equal(q[-n:].view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s[-n:], s1)
        del q
    g = hy.rms_norm_backward(y, h, w, rstd, dresidual_out=r)
    g1 = hy.rms_norm_backward(y[-n:], h1, w, rstd1, dresidual_out=r[-n:])
    assert torch.equal(g.dx[-n:], g1.dx) and torch.equal(g.dresidual[-n:], g1.dresidual)
    want, size = torch.zeros(D, dtype=torch.float64, device="cuda"), torch.zeros(D, dtype=torch.float64, device="cuda")
    for a in range(0, M, 8192):
        t = y[a:a + 8192].double() * h[a:a + 8192].double() * rstd[a:a + 8192, None].double()
        want += t.sum(0)
        size += t.abs().sum(0)
    # 148 CTAs' sums of about M / 148 rows, a step of 2^-24 each, and h rstd's rounding
    assert ((g.dweight.double() - want).abs() <= (M / 148 + 4) * 2.0 ** -24 * size).all()
