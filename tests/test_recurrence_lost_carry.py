"""What a look-back that runs out leaves in the results: NaN in all that the
missing carry reaches, the right values or NaN behind a reset, and the right
values in other channels and batch rows, which the carry has no part in.  The first unit's ticket
is taken away before the launch, so that no unit of the first chain is ever the
first; the wait gives up after about a second and the launch ends normally."""
import pytest

from .test_parity_recurrence import cuda, make, run_backward, run_forward, same

pytestmark = pytest.mark.gpu

L, D = 500, 64  # eight units, the last one of 52 tokens


def lost(hy, ws):
    with pytest.raises(hy.HyenaError) as err:
        hy.workspace_check(ws)
    assert err.value.status == 5  # HYENA_ERR_TIMEOUT
    hy.workspace_check(ws)  # reported once


@pytest.mark.parametrize("B", [1, 3])
def test_forward(B):
    import torch
    import hyena_long_convolution_b200 as hy
    c = cuda(make(B, L, D, seed=3))
    y, s, units = run_forward(hy, c, True)
    ws = hy.RecurrenceWorkspace(B, L, D)
    ws.buf[0] = 1  # header word 0, the next ticket: the first unit of batch row 0 is never run
    y2, s2, units2 = run_forward(hy, c, True, workspace=ws)
    lost(hy, ws)
    assert torch.isnan(y2[0, 64:]).all() and torch.isnan(s2[0]).all() and torch.isnan(units2[0, 1:]).all()
    assert same(y2[1:], y[1:]) and same(s2[1:], s[1:]) and same(units2[1:], units[1:])
    y2, s2, units2 = run_forward(hy, c, True, workspace=ws)
    assert same(y2, y) and same(s2, s) and same(units2, units)


def test_forward_with_resets():
    import torch
    import hyena_long_convolution_b200 as hy
    c = cuda(make(1, L, D, seed=4))
    c["reset"] = torch.zeros(1, L, dtype=torch.uint8, device="cuda")
    c["reset"][0, [70, 300]] = 2
    y, s, units = run_forward(hy, c, True)
    ws = hy.RecurrenceWorkspace(1, L, D)
    ws.buf[0] = 1
    y2, s2, units2 = run_forward(hy, c, True, workspace=ws)
    lost(hy, ws)
    assert torch.isnan(y2[0, 64:70]).all() and torch.isnan(units2[0, 1]).all()
    # what follows a reset in its unit needs no carry; the units behind have waited as
    # long as the one that the carry is missing from, and may have given up with it
    assert same(y2[0, 70:128], y[0, 70:128]) and same(y2[0, 300:320], y[0, 300:320])
    for got, want in ((y2[0, 64:], y[0, 64:]), (s2, s), (units2[0, 1:], units[0, 1:])):
        assert (torch.isnan(got) | (got == want)).all()


@pytest.mark.parametrize("B", [1, 3])
def test_gradient(B):
    import torch
    import hyena_long_convolution_b200 as hy
    c = cuda(make(B, L, D, seed=5))
    y, s, units = run_forward(hy, c, True)
    g = run_backward(hy, c, units, True)
    ws = hy.RecurrenceWorkspace(B, L, D)
    ws.buf[0] = 1  # the last unit of batch row 0
    g2 = run_backward(hy, c, units, True, workspace=ws)
    lost(hy, ws)
    last = L // 64 * 64
    for k in ("dx1", "dx2", "dgate"):
        got, want = getattr(g2, k), getattr(g, k)
        assert torch.isnan(got[0, :last]).all(), k
        assert same(got[1:], want[1:]), k
    assert same(g2.dx3[0, :last], g.dx3[0, :last]) and same(g2.dx3[1:], g.dx3[1:])
    assert torch.isnan(g2.dstate_in[0]).all() and same(g2.dstate_in[1:], g.dstate_in[1:])
    assert torch.isnan(g2.dlog_rate).all()
    g2 = run_backward(hy, c, units, True, workspace=ws)
    assert all(same(a, b) for a, b in zip(g2, g))
