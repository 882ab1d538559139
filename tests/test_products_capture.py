"""The products captured as programs capture them: calls that bring no workspace,
branches of a graph side by side, and replays one after another without a wait,
on inputs that change in between."""
import pytest

pytestmark = pytest.mark.gpu


def normal(*shape, seed, scale=1.0):
    import torch
    g = torch.Generator("cuda").manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)


class Block:
    """Weights of a block whose calls follow one another, and its buffers."""

    def __init__(self, M, D, F, seed):
        import hyena_long_convolution_b200 as hy
        self.x, self.dy = normal(M, D, seed=seed), normal(M, F, seed=seed + 1)
        self.wg, self.wu = (normal(F, D, seed=seed + i, scale=D ** -0.5) for i in (2, 3))
        self.qg, self.qu = (hy.fp8_quantize(w, block=128) for w in (self.wg, self.wu))
        self.down = hy.fp8_quantize(normal(D, F, seed=seed + 4, scale=F ** -0.5), block=128)

    def run(self):
        import torch
        import hyena_long_convolution_b200 as hy
        q, s = hy.fp8_quantize(self.x)
        fq, fs = hy.gated_ffn_fp8(q, s, *self.qg, *self.qu, "gelu", fp8_out=True)
        y = hy.fp8_matmul(fq, fs, *self.down)
        g, u = (torch.empty(*self.dy.shape, device="cuda") for _ in range(2))
        z = hy.gated_ffn(self.x, self.wg, self.wu, "silu", gate_out=g, up_out=u)
        d = hy.gated_ffn_backward(self.dy, self.x, self.wg, self.wu, g, u, "silu")
        return [y, z, g, u, *d]


SIZES = [(1, 264, 520), (40, 528, 1000), (300, 4400, 1664), (1000, 1032, 264)]


@pytest.mark.parametrize("M,D,F", SIZES)
def test_without_a_workspace(M, D, F):
    import torch
    b = Block(M, D, F, M)
    xs = [normal(M, D, seed=s) for s in range(4)]
    want = []
    for x in xs:
        b.x.copy_(x)
        want.append([t.clone() for t in b.run()])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = b.run()
    got = []
    for x in xs:
        b.x.copy_(x)
        graph.replay()
        got.append([t.clone() for t in out])
    for a, c in zip(want, got):
        assert all(torch.equal(t, v) for t, v in zip(a, c))


def test_branches_of_one_graph():
    """Two blocks on two streams of a graph, and a call that takes both results."""
    import torch
    import hyena_long_convolution_b200 as hy
    a, b = Block(300, 528, 1000, 1), Block(40, 528, 520, 5)

    def both(side):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            ob = b.run()
        oa = a.run()
        main.wait_stream(side)
        n = hy.gated_ffn(oa[0], a.wg, a.wu)  # of the one
        m = hy.gated_ffn(ob[0], a.wg, a.wu)  # and of the other
        return oa + ob + [n, m]

    side = torch.cuda.Stream()
    want = [t.clone() for t in both(side)]
    torch.cuda.synchronize()
    for _ in range(3):
        assert all(torch.equal(t, v) for t, v in zip(both(side), want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(side)
    for _ in range(5):
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        assert all(torch.equal(t, v) for t, v in zip(out, want))
