"""Failure detection of the gated recurrence's device-side waits, without a GPU
fault: the first unit's ticket is taken away before the launch, so that the
second unit looks back for one that never runs.  That wait gives up after about
a second, the launch ends normally, workspace_check reports HYENA_ERR_TIMEOUT,
and the same workspace then serves a correct call."""
import pytest

from .test_parity_recurrence import cuda, make, run_backward, run_forward, same

pytestmark = pytest.mark.gpu

TIMEOUT = 5  # HYENA_ERR_TIMEOUT


@pytest.mark.parametrize("back", [False, True])
def test_a_wait_runs_out_and_is_reported(back):
    import hyena_long_convolution_b200 as hy
    B, L, D = 1, 1000, 64
    c = cuda(make(B, L, D, seed=3))
    y, s, units = run_forward(hy, c, True)
    g = run_backward(hy, c, units, True)
    ws = hy.RecurrenceWorkspace(B, L, D)
    ws.buf[0] = 1  # header word 0: the next ticket
    run_backward(hy, c, units, True, workspace=ws) if back else run_forward(hy, c, True, workspace=ws)
    with pytest.raises(hy.HyenaError) as err:
        hy.workspace_check(ws)
    assert err.value.status == TIMEOUT
    y2, s2, units2 = run_forward(hy, c, True, workspace=ws)
    g2 = run_backward(hy, c, units2, True, workspace=ws)
    hy.workspace_check(ws)
    assert same(y, y2) and same(s, s2) and all(same(a, b) for a, b in zip(g, g2))
