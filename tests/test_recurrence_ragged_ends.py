"""The places behind a sequence's end in its last unit add nothing to the
gradients, whatever the last state is.  dlog_rate = sum of a q s_{t-1} sig takes
no part of the last token's own input where w = 1 (no normalisation), and none
of a reset's: with that input infinite, and with it the last state, it is bit
for bit what it is without."""
import pytest

from .test_parity_recurrence import cuda, make, run_backward, run_forward, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("L", [1, 7, 63, 64, 65, 72, 130])
@pytest.mark.parametrize("state", [True, False])
def test_an_infinite_last_state(L, normalize, state):
    import torch
    import hyena_long_convolution_b200 as hy
    c = cuda(make(2, L, 72, seed=L, state=state, resets="last" if normalize else None))
    _, _, units = run_forward(hy, c, normalize)
    g = run_backward(hy, c, units, normalize)
    d = dict(c, x1=c["x1"].clone())
    d["x1"][:, -1] = float("inf")
    _, s, units = run_forward(hy, d, normalize)
    assert torch.isinf(s).all()
    g2 = run_backward(hy, d, units, normalize)
    for k in ("dlog_rate", "dstate_in", "dgate", "dx1"):
        assert same(getattr(g2, k), getattr(g, k)), k
    assert same(g2.dx3[:, :-1], g.dx3[:, :-1]) and same(g2.dx2[:, :-1], g.dx2[:, :-1])
