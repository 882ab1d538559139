"""Cases of the 8-bit matrix product with scales per 128, its quantiser, and the
gated feed-forward block (bf16 with its gradient, and 8-bit): what they compute
in plain torch operations, the library's own calls, and what each pass cannot
do without.

Quantiser, per row and 128 channels (block 1) or per 128 x 128 block (block 128):
    scale = max(max |x|, 2^-100) / 448;  q = e4m3(x / scale)
Product of e4m3 tensors x [M, K] and w [N, K]:
    y[m, n] = sum_k (x[m, k] sx[m, k / 128]) (w[n, k] sw[n / 128, k / 128])
Gated feed-forward block, with x, gate and up weights in bf16 or as above:
    g = x Wg^T;  u = x Wu^T;  y = act(g) u     (bf16, or e4m3 with scales per 128)
    dg = dy u act'(g);  du = dy act(g)
    dx = dg Wg + du Wu;  dWg = dg^T x;  dWu = du^T x
"""
import math

import torch

own = False

E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100  # an all-zero group keeps a finite scale
ACTS = ("silu", "gelu", "gelu_tanh", "identity")
EXACT_FLOPS = 1e14  # about 3 s of 64-bit products


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one generated token's mixer output on its way into the output projection: launch latency
        dict(name="quantize_token", op="quantize", rows=1, D=4096, block=1, type="bf16"),
        # the mixer's output over a whole prompt of the headline length
        dict(name="quantize_prompt", op="quantize", rows=32768, D=4096, block=1, type="bf16"),
        # a feed-forward weight, once when a model is loaded
        dict(name="quantize_weight", op="quantize", rows=11008, D=4096, block=128, type="bf16"),
        # the input projection (x1, x2, x3 of 4096 channels) of one generated token, from the norm's one scale a row
        dict(name="matmul_token", op="matmul", M=1, K=4096, N=12288, group=0, out="bf16"),
        # the down projection of 64 sequences decoded together
        dict(name="matmul_batch", op="matmul", M=64, K=11008, N=4096, group=128, out="bf16"),
        # the input projection of an 8K prompt
        dict(name="matmul_8k", op="matmul", M=8192, K=4096, N=12288, group=128, out="bf16"),
        # odd rows, widths that fill no whole tile and a K that ends inside a block, fp32 output
        dict(name="matmul_ragged", op="matmul", M=999, K=1040, N=1032, group=128, out="fp32"),
        # one generated token through the feed-forward block in bf16
        dict(name="ffn_token", op="ffn", do="forward", M=1, D=4096, F=11008, act="silu"),
        # a training step's forward and backward over 8K tokens
        dict(name="ffn_train_8k", op="ffn", do="train", M=8192, D=4096, F=11008, act="silu", keep="fp32"),
        # the same over packed documents of odd lengths in a small model of odd widths
        dict(name="ffn_train_ragged", op="ffn", do="train", M=1000, D=1032, F=2760, act="gelu", keep="fp32"),
        # 16 sequences decoded together, codes out for the down projection
        dict(name="ffn_fp8_batch", op="ffn_fp8", M=16, D=4096, F=11008, act="silu", group=128, out="fp8"),
        # one 1024-token chunk of a chunked prefill
        dict(name="ffn_fp8_chunk", op="ffn_fp8", M=1024, D=4096, F=11008, act="gelu", group=128, out="fp8"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    def width(lo, hi, step):
        return max(lo, step * (_spread(rng, lo, hi) // step))

    op = rng.choice(["quantize", "matmul", "matmul", "ffn", "ffn", "ffn_fp8"])
    if op == "quantize":
        c = dict(op=op, rows=_spread(rng, 1, 65536), D=width(64, 16384, 8), block=rng.choice([1, 128]),
                 type=rng.choice(["bf16", "fp32"]))
        while c["rows"] * c["D"] > 2 ** 28:
            c["rows"] = c["rows"] * 2 // 3
        return c
    M = _spread(rng, 1, 8192)
    if op == "matmul":
        c = dict(op=op, M=M, K=width(64, 16384, 16), N=width(64, 16384, 8), group=rng.choice([0, 128]),
                 out=rng.choice(["bf16", "bf16", "fp32"]))
    elif op == "ffn":
        c = dict(op=op, do=rng.choice(["forward", "train"]), M=M, D=width(64, 8192, 8), F=width(64, 16384, 8),
                 act=rng.choice(ACTS))
        if c["do"] == "train":
            c["keep"] = rng.choice(["bf16", "fp32"])
    else:
        c = dict(op=op, M=M, D=width(64, 8192, 16), F=width(64, 16384, 16), act=rng.choice(ACTS),
                 group=rng.choice([0, 128]), out=rng.choice(["bf16", "fp8"]))
    most = 12 * 8192 * 4096 * 11008  # the largest listed case
    while work(c)["flops"] > most:
        c["M"] = c["M"] * 2 // 3
    return c


def _groups(n):
    return -(-n // 128)


def work(case):
    c = case
    if c["op"] == "quantize":
        n = c["rows"] * c["D"]
        rows = c["rows"] if c["block"] == 1 else _groups(c["rows"])
        return {"bytes": n * ((2 if c["type"] == "bf16" else 4) + 1) + 4 * rows * _groups(c["D"]), "flops": 3 * n}
    M = c["M"]
    if c["op"] == "matmul":
        K, N = c["K"], c["N"]
        scales = M * (_groups(K) if c["group"] else 1) + _groups(N) * _groups(K)
        return {"bytes": M * K + N * K + 4 * scales + M * N * (2 if c["out"] == "bf16" else 4), "flops": 2 * M * N * K}
    D, F = c["D"], c["F"]
    if c["op"] == "ffn_fp8":
        scales = M * (_groups(D) if c["group"] else 1) + 2 * _groups(F) * _groups(D)
        scales += M * _groups(F) if c["out"] == "fp8" else 0
        return {"bytes": M * D + 2 * F * D + 4 * scales + M * F * (1 if c["out"] == "fp8" else 2),
                "flops": 4 * M * F * D}
    if c["do"] == "forward":
        return {"bytes": 2 * M * D + 4 * F * D + 2 * M * F, "flops": 4 * M * F * D}
    # x, the weights and dy in; y, dx and the weights' gradients out
    return {"bytes": 4 * M * D + 8 * F * D + 4 * M * F, "flops": 12 * M * F * D}


# ----------------------------------------------------------------- inputs

def _codes(x, block):
    """(q, scales) of x by groups of `block` rows x 128 channels."""
    R, C = x.shape
    r, g = -(-R // block), _groups(C)
    p = x.new_zeros(r * block, g * 128)
    p[:R, :C] = x
    p = p.view(r, block, g, 128)
    scales = torch.clamp(p.abs().amax((1, 3)), min=AMAX_FLOOR) / E4M3_MAX
    q = torch.clamp(p / scales[:, None, :, None], -E4M3_MAX, E4M3_MAX).view(r * block, g * 128)[:R, :C]
    return q.to(torch.float8_e4m3fn), scales


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * scale

    def activations(rows, width):
        # channels of different sizes, as a norm's weight and a mixer leave them
        return normal(rows, width) * torch.exp(0.5 * normal(width))

    def weight(n, k):
        # rows of different sizes; products of about unit size
        return normal(n, k) * torch.exp(0.3 * normal(n, 1)) * k ** -0.5

    s = dict(case=c)
    if c["op"] == "quantize":
        x = activations(c["rows"], c["D"]) if c["block"] == 1 else weight(c["rows"], c["D"])
        s["x"] = x.to(torch.bfloat16) if c["type"] == "bf16" else x
        return s
    M = c["M"]
    if c["op"] == "ffn":
        D, F = c["D"], c["F"]
        s["x"] = normal(M, D).to(torch.bfloat16)
        s["gate"], s["up"] = weight(F, D).to(torch.bfloat16), weight(F, D).to(torch.bfloat16)
        if c["do"] == "train":
            s["dy"] = normal(M, F).to(torch.bfloat16)
    else:
        K = c["K"] if c["op"] == "matmul" else c["D"]
        x = activations(M, K)
        if c["group"]:
            s["x"], s["sx"] = _codes(x, 1)
        else:  # one scale a row
            s["sx"] = x.abs().amax(1, keepdim=True) / E4M3_MAX
            s["x"] = (x / s["sx"]).to(torch.float8_e4m3fn)
        if c["op"] == "matmul":
            s["w"], s["sw"] = _codes(weight(c["N"], K), 128)
        else:
            s["gate"], s["sgate"] = _codes(weight(c["F"], K), 128)
            s["up"], s["sup"] = _codes(weight(c["F"], K), 128)
    if own:
        import hyena_long_convolution_b200 as hy
        if c["op"] == "matmul":
            s["workspace"] = hy.MatmulWorkspace(M, c["N"], c["K"])
        else:
            s["workspace"] = hy.FfnWorkspace(M, c["D"], c["F"], backward=c.get("do") == "train")
    return s


def run(state):
    c = state["case"]
    if own:
        return {"quantize": _own_quantize, "matmul": _own_matmul, "ffn": _own_ffn, "ffn_fp8": _own_ffn_fp8}[c["op"]](state)
    return {"quantize": _plain_quantize, "matmul": _plain_matmul, "ffn": _plain_ffn,
            "ffn_fp8": _plain_ffn_fp8}[c["op"]](state)


# ------------------------------------------------------- the library's calls

def _own_quantize(s):
    import hyena_long_convolution_b200 as hy
    q, scales = hy.fp8_quantize(s["x"], block=s["case"]["block"])
    return dict(q=q, scales=scales)


def _own_matmul(s):
    import hyena_long_convolution_b200 as hy
    dtype = torch.bfloat16 if s["case"]["out"] == "bf16" else torch.float32
    return dict(y=hy.fp8_matmul(s["x"], s["sx"], s["w"], s["sw"], dtype=dtype, workspace=s["workspace"]))


def _own_ffn(s):
    import hyena_long_convolution_b200 as hy
    c, x = s["case"], s["x"]
    if c["do"] == "forward":
        return dict(y=hy.gated_ffn(x, s["gate"], s["up"], c["act"], workspace=s["workspace"]))
    kept = torch.bfloat16 if c["keep"] == "bf16" else torch.float32
    g = torch.empty(c["M"], c["F"], dtype=kept, device="cuda")
    u = torch.empty_like(g)
    y = hy.gated_ffn(x, s["gate"], s["up"], c["act"], gate_out=g, up_out=u, workspace=s["workspace"])
    d = hy.gated_ffn_backward(s["dy"], x, s["gate"], s["up"], g, u, c["act"], workspace=s["workspace"])
    return dict(y=y, dx=d.dx, dgate=d.dgate_weight, dup=d.dup_weight)


def _own_ffn_fp8(s):
    import hyena_long_convolution_b200 as hy
    c = s["case"]
    y = hy.gated_ffn_fp8(s["x"], s["sx"], s["gate"], s["sgate"], s["up"], s["sup"], c["act"],
                         fp8_out=c["out"] == "fp8", workspace=s["workspace"])
    return dict(q=y[0], scales=y[1]) if c["out"] == "fp8" else dict(y=y)


# ------------------------------------------------------------- plain forms

def _values(q, scales, block):
    """The fp32 values that codes with scales per `block` rows x 128 channels (or one a row) stand for."""
    s = scales if block == 1 else scales.repeat_interleave(block, 0)[:q.shape[0]]
    return q.float() * (s if s.shape[1] == 1 else s.repeat_interleave(128, 1)[:, :q.shape[1]])


def _act(name, g):
    """(act(g), act'(g))."""
    if name == "identity":
        return g, torch.ones_like(g)
    if name == "silu":
        sig = 1.0 / (1.0 + torch.exp(-g))
        return g * sig, sig * (1.0 + g * (1.0 - sig))
    if name == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (0.5 / math.pi) ** 0.5
    k, cubic = (2.0 / math.pi) ** 0.5, 0.044715
    t = torch.tanh(k * (g + cubic * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * k * (1.0 + 3.0 * cubic * g * g)


def _plain_quantize(s):
    q, scales = _codes(s["x"].float(), s["case"]["block"])
    return dict(q=q, scales=scales)


def _plain_matmul(s):
    y = _values(s["x"], s["sx"], 1) @ _values(s["w"], s["sw"], 128).t()
    return dict(y=y.to(torch.bfloat16) if s["case"]["out"] == "bf16" else y)


def _plain_ffn(s):
    c, b = s["case"], torch.bfloat16
    x, wg, wu = s["x"].float(), s["gate"].float(), s["up"].float()
    g, u = x @ wg.t(), x @ wu.t()
    a, da = _act(c["act"], g)
    y = (a * u).to(b)
    if c["do"] == "forward":
        return dict(y=y)
    dy = s["dy"].float()
    dg, du = dy * u * da, dy * a
    return dict(y=y, dx=(dg @ wg + du @ wu).to(b), dgate=(dg.t() @ x).to(b), dup=(du.t() @ x).to(b))


def _plain_ffn_fp8(s):
    c, x = s["case"], _values(s["x"], s["sx"], 1)
    a, _ = _act(c["act"], x @ _values(s["gate"], s["sgate"], 128).t())
    y = a * (x @ _values(s["up"], s["sup"], 128).t())
    if c["out"] == "bf16":
        return dict(y=y.to(torch.bfloat16))
    q, scales = _codes(y, 1)
    return dict(q=q, scales=scales)


# ------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    if work(case)["flops"] > EXACT_FLOPS:
        return None
    s = prepare(case, seed)
    c, f64 = s["case"], torch.float64

    def wide(q, scales, block):
        R, C = q.shape
        v = q.to(f64)
        if scales.shape[1] == 1 and block == 1:
            return v * scales.to(f64)
        for i in range(_groups(C)):
            col = scales[:, i].to(f64)
            v[:, i * 128:(i + 1) * 128] *= torch.repeat_interleave(col, block)[:R, None]
        return v

    def quotients(y, block):
        bands = [torch.stack([p.abs().max() for p in rows.split(128, 1)]) if block > 1 else
                 torch.stack([p.abs().max(1).values for p in rows.split(128, 1)], 1)
                 for rows in (y.split(block, 0) if block > 1 else [y])]
        scales = (torch.stack(bands) if block > 1 else bands[0]).clamp_min(AMAX_FLOOR) / E4M3_MAX
        at = torch.arange(y.shape[0], device=y.device) // block, torch.arange(y.shape[1], device=y.device) // 128
        return dict(q=y / scales[at[0]][:, at[1]], scales=scales)

    if c["op"] == "quantize":
        return quotients(s["x"].to(f64), c["block"])
    if c["op"] == "matmul":
        return dict(y=torch.matmul(wide(s["x"], s["sx"], 1), wide(s["w"], s["sw"], 128).T))
    train = c.get("do") == "train"
    if c["op"] == "ffn":
        x, wg, wu = (s[k].to(f64).requires_grad_(train) for k in ("x", "gate", "up"))
    else:
        x = wide(s["x"], s["sx"], 1)
        wg, wu = wide(s["gate"], s["sgate"], 128), wide(s["up"], s["sup"], 128)
    g = torch.matmul(x, wg.T)
    fn = torch.nn.functional
    act = {"silu": fn.silu, "gelu": fn.gelu, "gelu_tanh": lambda v: fn.gelu(v, approximate="tanh"),
           "identity": lambda v: v}[c["act"]]
    y = act(g) * torch.matmul(x, wu.T)
    if c["op"] == "ffn_fp8" and c["out"] == "fp8":
        return quotients(y, 1)
    out = dict(y=y.detach())
    if train:
        y.backward(s["dy"].to(f64))
        out.update(dx=x.grad, dgate=wg.grad, dup=wu.grad)
    return out
