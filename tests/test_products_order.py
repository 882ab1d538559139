"""Quantiser and product in turn on the same buffers, with other data every turn:
each kernel is launched while the one ahead of it ends, and one that read its
inputs too soon, or let them be written too soon, would work on another turn's."""
import pytest

pytestmark = pytest.mark.gpu


# by rows and width: one CTA a tile; clusters of two and of four; pairs with whole tiles, pairs
# that share a tile's k; single CTAs that share it
@pytest.mark.parametrize("M,D", [(2, 256), (16, 1032), (16, 4096), (2100, 520), (300, 4400), (128, 9488)])
def test_each_turn_works_on_its_own_data(M, D):
    import torch
    import hyena_long_convolution_b200 as hy
    g = torch.Generator("cuda").manual_seed(M)
    turns = 8
    xs = [torch.randn(M, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(turns)]
    w1, w2 = (hy.fp8_quantize((torch.randn(D, D, generator=g, device="cuda") * D ** -0.5).to(torch.bfloat16), block=128)
              for _ in range(2))
    ws = hy.MatmulWorkspace(M, D, D)
    q = torch.zeros(M, -(-D // 16) * 16, device="cuda").to(torch.float8_e4m3fn)[:, :D]
    s = torch.empty(M, -(-D // 128), device="cuda")
    y = torch.empty(M, D, dtype=torch.bfloat16, device="cuda")

    def turn(x, z, after):
        for call in (lambda: hy.fp8_quantize(x, q=q, scales=s), lambda: hy.fp8_matmul(q, s, *w1, y=y, workspace=ws),
                     lambda: hy.fp8_quantize(y, q=q, scales=s), lambda: hy.fp8_matmul(q, s, *w2, y=z, workspace=ws)):
            call()
            after()

    want = [torch.empty_like(y) for _ in xs]
    for x, z in zip(xs, want):
        turn(x, z, torch.cuda.synchronize)
    assert all(torch.isfinite(z).all() for z in want) and not torch.equal(want[0], want[1])
    for _ in range(5):
        got = [torch.full_like(y, float("nan")) for _ in xs]
        for t in (q.view(torch.uint8), s, y):
            t.fill_(0x7f if t.dtype is torch.uint8 else float("nan"))
        torch.cuda.synchronize()
        for x, z in zip(xs, got):
            turn(x, z, lambda: None)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    hy.workspace_check(ws)
