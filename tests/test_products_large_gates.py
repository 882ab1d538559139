"""The gradient of the gated feed-forward block at large finite gates, where an
activation's slope is 1 or 0 and the squares and cubes on the way to it overflow."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "identity"])
def test_slopes_of_large_gates(act):
    """From |g| = 200 on act(g) is g or 0 and act'(g) 1 or 0, to the last bit of fp32."""
    import torch
    import hyena_long_convolution_b200 as hy
    big = [200.0, 1e4, 1e10, 1.5e19, 1.9e19, 1e25, 1e38, 3e38]
    g = torch.tensor([big, [-v for v in big]], device="cuda")
    one = torch.ones(2, 8, device="cuda")
    eye, none = torch.eye(8), torch.zeros(8, 8)
    wg, wu = (torch.cat(p, 1).to(torch.bfloat16).cuda() for p in ((eye, none), (none, eye)))  # dx = [dg | du]
    x = torch.zeros(2, 16, dtype=torch.bfloat16, device="cuda")
    for keep in (torch.float32, torch.bfloat16):
        kept = g.to(keep)
        dx = hy.gated_ffn_backward(one.bfloat16(), x, wg, wu, kept, one.to(keep), act).dx
        on = torch.ones_like(g) if act == "identity" else (g > 0).float()
        assert torch.equal(dx[:, :8].float(), on), act
        assert torch.equal(dx[:, 8:].float(), torch.where(on > 0, kept.float(), on).bfloat16().float()), act
