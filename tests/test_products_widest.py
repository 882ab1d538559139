"""The products' largest widths, on whole numbers that every order of summation
holds exactly."""
import pytest

pytestmark = pytest.mark.gpu

MOST = 1 << 20


def whole(*shape, seed, top=1):
    import torch
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=g, device="cuda").float()


@pytest.mark.parametrize("M,N,K", [(1, 8, MOST), (3, MOST, 24), (40, 136, MOST), (20, MOST, 136), (300, MOST, 8),
                                   (300, 16, MOST)])
def test_matmul(M, N, K):
    import torch
    import hyena_long_convolution_b200 as hy
    x, w = whole(M, K, seed=1), whole(N, K, seed=2)

    def codes(t, block):  # ones and zeros are codes, scaled by 1
        q = torch.zeros(t.shape[0], -(-K // 16) * 16, device="cuda").to(torch.float8_e4m3fn)[:, :K]
        q.copy_(t.to(torch.float8_e4m3fn))
        return q, torch.ones(-(-t.shape[0] // block), -(-K // 128), device="cuda")

    y = hy.fp8_matmul(*codes(x, 1), *codes(w, 128), dtype=torch.float32)
    assert torch.equal(y, (x.double() @ w.double().T).float())


@pytest.mark.parametrize("M,D,F", [(3, 8, MOST), (200, 8, MOST), (3, MOST, 8), (200, MOST, 8)])
def test_ffn_and_its_gradient(M, D, F):
    """Identity for the activation: y = g u, and with g and u of -1, 0 and 1 dg = dy u, du = dy g."""
    import torch
    import hyena_long_convolution_b200 as hy
    b = torch.bfloat16
    x, wg, wu = whole(M, D, seed=1), whole(F, D, seed=2), whole(F, D, seed=3)
    g, u, dy = (whole(M, F, seed=s) for s in (4, 5, 6))
    kept = [torch.empty(M, F, device="cuda") for _ in range(2)]
    y = hy.gated_ffn(x.to(b), wg.to(b), wu.to(b), "identity", gate_out=kept[0], up_out=kept[1])
    rg, ru = ((x.double() @ w.double().T).float() for w in (wg, wu))
    assert torch.equal(kept[0], rg) and torch.equal(kept[1], ru) and torch.equal(y, (rg * ru).to(b))
    d = hy.gated_ffn_backward(dy.to(b), x.to(b), wg.to(b), wu.to(b), g, u, "identity")
    dg, du = (dy * u).double(), (dy * g).double()
    # sums below 2^24, rounded once
    assert torch.equal(d.dx, (dg @ wg.double() + du @ wu.double()).float().to(b))
    assert torch.equal(d.dgate_weight, (dg.T @ x.double()).float().to(b))
    assert torch.equal(d.dup_weight, (du.T @ x.double()).float().to(b))


@pytest.mark.parametrize("rows,D,block", [(3, MOST, 1), (130, MOST, 128), (1 << 20, 8, 1)])
def test_quantize(rows, D, block):
    """Whole numbers up to 7 with one of 448 in each group are their own codes."""
    import torch
    import hyena_long_convolution_b200 as hy
    x = whole(rows, D, seed=3, top=7)
    x[::block, ::128] = 448.0
    q, s = hy.fp8_quantize(x, block=block)
    assert (s == 1.0).all() and torch.equal(q.float(), x)
