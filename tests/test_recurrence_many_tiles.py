"""The gated recurrence with many more tiles than CTAs on the device, each CTA
going through several of them: sequences of one unit, where no carry is looked
for and the next rows are asked for at the last moment, and of two.  Against
the fp64 oracle with the bounds of test_parity_recurrence."""
import pytest

from .test_parity_recurrence import check, cuda, make, run_backward, run_forward, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("B,L,D,resets", [
    (64, 40, 2048, None),    # 2048 tiles of one unit
    (64, 40, 2048, 0.1),
    (300, 64, 320, None),    # 1500, whole units
    (512, 1, 256, None),     # 2048 of one token
    (40, 70, 1024, 0.02),    # 1280 of two units, the second one of six tokens
])
def test_matches_oracle(B, L, D, resets, normalize):
    import hyena_long_convolution_b200 as hy
    d = make(B, L, D, seed=B + L + D, resets=resets)
    c = cuda(d)
    ws = hy.RecurrenceWorkspace(B, L, D)
    y, s, units = run_forward(hy, c, normalize, workspace=ws)
    g = run_backward(hy, c, units, normalize, workspace=ws)
    hy.workspace_check(ws)
    check(d, normalize, y, s, units, g)


@pytest.mark.parametrize("B,L,D", [(64, 40, 2048), (40, 70, 1024)])
def test_states_and_their_gradients_in_place(B, L, D):
    """state_out may be state_in and dstate_in dstate_out, call after call."""
    import hyena_long_convolution_b200 as hy
    c = cuda(make(B, L, D, seed=7))
    ws = hy.RecurrenceWorkspace(B, L, D)
    y, s, units = run_forward(hy, c, True, workspace=ws)
    g = run_backward(hy, c, units, True, workspace=ws)
    fwd = [c[k] for k in ("x1", "x2", "x3", "gate", "log_rate", "Dskip")]
    for _ in range(5):
        S, e = c["state_in"].clone(), c["dstate_out"].clone()
        y2 = hy.gated_recurrence(*fwd, state_in=S, state_out=S, workspace=ws)
        g2 = hy.gated_recurrence_backward(c["dy"], *fwd, units, dstate_out=e, dstate_in=e, workspace=ws)
        assert same(y2, y) and same(S, s) and same(e, g.dstate_in)
        assert all(same(a, b) for a, b in zip(g2, g))
    hy.workspace_check(ws)
