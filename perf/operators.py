"""Cases of the gated linear recurrence (forward, backward, decode) and of the
root-mean-square norm with the residual's addition (bf16 and 8-bit outputs,
backward): what they compute in plain torch operations, the library's own
calls, and what each pass cannot do without.

Gated linear recurrence, per channel, with v = x1 x2:
    a_t = exp(log_rate * sigmoid(gate_t))  (0 where reset_t)
    s_t = a_t s_{t-1} + w_t v_t,   w_t = sqrt(1 - a_t^2) (normalize) or 1
    y_t = x3_t s_t + Dskip v_t
Norm over the channels of each row:
    h = x + residual, held in the residual's type;  n = h / sqrt(mean(h^2) + eps)
    y = n weight, in bf16, or as e4m3 values with one scale per row or per 128 channels
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100  # an all-zero row or group keeps a finite scale


# ------------------------------------------------------------------ cases

def listed():
    rec, norm = "recurrence", "norm"
    return [
        # one generated token of one sequence, at the library's 4096 channels: launch latency
        dict(name="decode_b1", op=rec, do="decode", B=1, L=1, D=4096, normalize=True, skip=True),
        # one generated token of 64 sequences served together
        dict(name="decode_b64", op=rec, do="decode", B=64, L=1, D=4096, normalize=False, skip=True),
        # one 1024-token chunk of a chunked prefill, state carried in and out
        dict(name="chunk_1k", op=rec, do="forward", B=1, L=1024, D=4096, normalize=True, skip=True, reset=False,
             state=True),
        # a whole prompt of the headline length in a single pass
        dict(name="prefill_32k", op=rec, do="forward", B=1, L=32768, D=4096, normalize=True, skip=True, reset=False,
             state=False),
        # a training step's forward and backward at the 8K context, two sequences
        dict(name="train_8k", op=rec, do="train", B=2, L=8192, D=4096, normalize=True, skip=True, reset=False,
             state=False),
        # packed documents of odd lengths (reset at each start), a width that fills no whole tile, no skip,
        # a state carried in and its gradient carried out, as in truncated backpropagation
        dict(name="train_ragged", op=rec, do="train", B=3, L=1000, D=1032, normalize=False, skip=False, reset=True,
             state=True),
        # the norm before the projection of one generated token, in 8 bits with a scale for the row
        dict(name="norm_decode_fp8", op=norm, do="fp8", rows=1, D=4096, group=0, res="bf16"),
        # the norm of a whole 32K prompt over a bf16 residual stream
        dict(name="norm_32k", op=norm, do="bf16", rows=32768, D=4096, res="bf16"),
        # the norm of an 8K prompt over an fp32 residual stream, in 8 bits with a scale per 128 channels
        dict(name="norm_fp8_8k", op=norm, do="fp8", rows=8192, D=4096, group=128, res="fp32"),
        # the norm's forward and backward in a training step of two 8K sequences
        dict(name="norm_train_8k", op=norm, do="train", rows=16384, D=4096, res="bf16"),
        # odd rows of a width that fills no whole vector block, an fp32 residual stream, forward and backward
        dict(name="norm_train_ragged", op=norm, do="train", rows=999, D=1032, res="fp32"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = 1.3e9  # bytes: the largest listed cases' and no more
    kind = rng.choice(["decode", "forward", "forward", "train", "train", "fp8", "bf16", "norm_train"])
    D = max(64, 8 * (_spread(rng, 64, 8192) // 8))
    if kind in ("fp8", "bf16", "norm_train"):
        c = dict(op="norm", do="train" if kind == "norm_train" else kind, rows=_spread(rng, 1, 32768), D=D,
                 res=rng.choice(["bf16", "fp32", "none"]))
        if kind == "fp8":
            c["group"] = rng.choice([0, 128])
        while work(c)["bytes"] > most:
            c["rows"] = c["rows"] * 2 // 3
        return c
    c = dict(op="recurrence", do=kind, B=_spread(rng, 1, 8), L=_spread(rng, 1, 32768), D=D,
             normalize=rng.random() < 0.5, skip=rng.random() < 0.5)
    if kind == "decode":
        c["B"], c["L"] = _spread(rng, 1, 256), 1
    else:
        c["reset"], c["state"] = rng.random() < 0.3, rng.random() < 0.5
    while work(c)["bytes"] > most:
        c["L"] = c["L"] * 2 // 3
    return c


def work(case):
    c = case
    if c["op"] == "norm":
        n, D = c["rows"] * c["D"], c["D"]
        r = {"bf16": 2, "fp32": 4, "none": 0}[c["res"]]
        fwd = n * (2 + 2 * r + 2) + 4 * D
        if c["do"] == "fp8":
            groups = c["rows"] * (1 if c["group"] == 0 else -(-D // c["group"]))
            return {"bytes": n * (2 + 2 * r + 1) + 4 * D + 4 * groups, "flops": 7 * n}
        if c["do"] == "bf16":
            return {"bytes": fwd, "flops": 5 * n}
        # backward: dy, h, the residual's gradient in; dx (and the fp32 residual's gradient) out
        h = r if r else 2
        bwd = n * (2 + h + r + 2 + (4 if c["res"] == "fp32" else 0)) + 8 * D + 4 * c["rows"]
        return {"bytes": fwd + 4 * c["rows"] + bwd, "flops": 16 * n}
    n, D = c["B"] * c["L"] * c["D"], c["D"]
    par = 8 * D
    if c["do"] == "decode":
        return {"bytes": n * 18 + par, "flops": 16 * n}
    resets = c["B"] * c["L"] if c["reset"] else 0
    fwd = 10 * n + par + resets + c["B"] * D * (4 + 4 * c["state"])
    if c["do"] == "forward":
        return {"bytes": fwd, "flops": 16 * n}
    bwd = 18 * n + par + 8 * D + resets + c["B"] * D * (4 + 4 * c["state"])
    return {"bytes": fwd + bwd, "flops": 56 * n}


# ----------------------------------------------------------------- inputs

def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, dtype=torch.bfloat16, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    if c["op"] == "norm":
        M, D = c["rows"], c["D"]
        s = dict(case=c, x=normal(M, D), weight=1.0 + normal(D, dtype=torch.float32, scale=0.1), residual=None)
        if c["res"] != "none":
            s["residual"] = normal(M, D, dtype=torch.bfloat16 if c["res"] == "bf16" else torch.float32, scale=4.0)
        if c["do"] == "train":
            s["dy"] = normal(M, D)
            s["dh"] = None if s["residual"] is None else normal(M, D).to(s["residual"].dtype)
        return s
    B, L, D = c["B"], c["L"], c["D"]
    # log rates: the library's draw of log poles, -exp(U(ln 1e-3, 0))
    lr = -torch.exp(torch.rand(D, generator=gen, device="cuda") * math.log(1e3) + math.log(1e-3))
    s = dict(case=c, x1=normal(B, L, D), x2=normal(B, L, D), x3=normal(B, L, D), gate=normal(B, L, D, scale=1.5),
             log_rate=lr, Dskip=normal(D, dtype=torch.float32) if c["skip"] else None)
    if c["do"] == "decode":
        s["state"] = normal(B, D, dtype=torch.float32)
        for k in ("x1", "x2", "x3", "gate"):
            s[k] = s[k][:, 0]
        return s
    s["state_in"] = normal(B, D, dtype=torch.float32) if c["state"] else None
    # documents of about 300 tokens
    s["reset"] = (torch.rand(B, L, generator=gen, device="cuda") < 1 / 300) if c["reset"] else None
    if c["do"] == "train":
        s["dy"] = normal(B, L, D)
        s["dstate_out"] = normal(B, D, dtype=torch.float32) if c["state"] else None
    if own:
        import hyena_long_convolution_b200 as hy
        s["workspace"] = hy.RecurrenceWorkspace(B, L, D)
    return s


def run(state):
    c = state["case"]
    if own:
        return _own_norm(state) if c["op"] == "norm" else _own_recurrence(state)
    return _plain_norm(state) if c["op"] == "norm" else _plain_recurrence(state)


# ------------------------------------------------------- the library's calls

def _own_recurrence(s):
    import hyena_long_convolution_b200 as hy
    c = s["case"]
    if c["do"] == "decode":
        y = hy.gated_recurrence_decode(s["x1"], s["x2"], s["x3"], s["gate"], s["log_rate"], s["Dskip"], s["state"],
                                       normalize=c["normalize"])
        return dict(y=y, state=s["state"])
    B, L, D = c["B"], c["L"], c["D"]
    state_out = torch.empty(B, D, device="cuda")
    units = hy.recurrence_unit_states(B, L, D, device="cuda") if c["do"] == "train" else None
    y = hy.gated_recurrence(s["x1"], s["x2"], s["x3"], s["gate"], s["log_rate"], s["Dskip"], reset=s["reset"],
                            normalize=c["normalize"], state_in=s["state_in"], state_out=state_out, unit_states=units,
                            workspace=s["workspace"])
    out = dict(y=y, state_out=state_out)
    if c["do"] == "train":
        g = hy.gated_recurrence_backward(s["dy"], s["x1"], s["x2"], s["x3"], s["gate"], s["log_rate"], s["Dskip"],
                                         units, reset=s["reset"], normalize=c["normalize"],
                                         dstate_out=s["dstate_out"], workspace=s["workspace"])
        out.update(dx1=g.dx1, dx2=g.dx2, dx3=g.dx3, dgate=g.dgate, dlog_rate=g.dlog_rate, dDskip=g.dDskip,
                   dstate_in=g.dstate_in if c["state"] else None)
    return out


def _own_norm(s):
    import hyena_long_convolution_b200 as hy
    c, x, res = s["case"], s["x"], s["residual"]
    h = None if res is None else torch.empty_like(res)
    if c["do"] == "fp8":
        q, scales = hy.rms_norm_fp8(x, s["weight"], EPS, residual=res, residual_out=h, group=c["group"])
        return dict(q=q, scales=scales, h=h)
    if c["do"] == "bf16":
        return dict(y=hy.rms_norm(x, s["weight"], EPS, residual=res, residual_out=h), h=h)
    rstd = torch.empty(x.shape[0], device="cuda")
    y = hy.rms_norm(x, s["weight"], EPS, residual=res, residual_out=h, rstd=rstd)
    g = hy.rms_norm_backward(s["dy"], x if h is None else h, s["weight"], rstd, dresidual_out=s["dh"])
    return dict(y=y, h=h, dx=g.dx, dresidual=g.dresidual if c["res"] == "fp32" else None, dweight=g.dweight)


# ------------------------------------------------------------- plain forms

def _scan(a, u):
    """(prefix products of a, states of s_t = a_t s_{t-1} + u_t from zero) along dim 1, by doubling: log2(L) steps."""
    k = 1
    while k < u.shape[1]:
        u = torch.cat((u[:, :k], u[:, k:] + a[:, k:] * u[:, :-k]), 1)
        a = torch.cat((a[:, :k], a[:, k:] * a[:, :-k]), 1)
        k *= 2
    return a, u


def _gates(s):
    """sigmoid, decay (0 at resets) and input weight of every token.

    In 64 bits, as the scans over them: slow channels decay by 1e-3 a token or less, so that 32 bits round the
    decay next to 1 and multiply the error over thousands of tokens."""
    sig = 1.0 / (1.0 + torch.exp(-s["gate"].double()))
    l = s["log_rate"] * sig
    a, z = torch.exp(l), -torch.expm1(2.0 * l)
    if s.get("reset") is not None:
        keep = (s["reset"] == 0)[..., None]
        a, z = a * keep, torch.where(keep, z, torch.ones_like(z))
    return sig, a, torch.sqrt(z) if s["case"]["normalize"] else None


def _plain_recurrence(s):
    c = s["case"]
    x1, x2, x3 = s["x1"].float(), s["x2"].float(), s["x3"].float()
    D = s["Dskip"]
    sig, a, w = _gates(s)
    v = x1 * x2
    u = v if w is None else w * v
    if c["do"] == "decode":
        h = a * s["state"] + u
        s["state"].copy_(h)
        y = x3 * h
        return dict(y=(y if D is None else y + D * v).to(torch.bfloat16), state=s["state"])
    pa, st = _scan(a, u)
    if s["state_in"] is not None:
        st = st + pa * s["state_in"][:, None]
    y = x3 * st
    out = dict(y=(y if D is None else y + D * v).to(torch.bfloat16), state_out=st[:, -1].float())
    if c["do"] == "forward":
        return out
    dy = s["dy"].float()
    # q_t = x3_t dy_t + a_{t+1} q_{t+1}: the same scan over the reversed axis
    r = x3 * dy
    an = torch.cat((a[:, 1:], torch.ones_like(a[:, :1])), 1)
    pq, q = _scan(an.flip(1), r.flip(1))
    if s["dstate_out"] is not None:
        q = q + pq * s["dstate_out"][:, None]
    q = q.flip(1)
    first = torch.zeros_like(st[:, :1]) if s["state_in"] is None else s["state_in"][:, None]
    prev = torch.cat((first, st[:, :-1]), 1)
    dl = a * q * prev
    if w is not None:
        dl = dl - q * v * a * a / w
    dv = q if w is None else w * q
    if D is not None:
        dv = dv + D * dy
        out["dDskip"] = (dy * v).sum((0, 1), dtype=torch.float64).float()
    else:
        out["dDskip"] = None
    b = torch.bfloat16
    out.update(dx1=(dv * x2).to(b), dx2=(dv * x1).to(b), dx3=(dy * st).to(b),
               dgate=(dl * s["log_rate"] * sig * (1.0 - sig)).to(b),
               dlog_rate=(dl * sig).sum((0, 1)).float(),
               dstate_in=(a[:, 0] * q[:, 0]).float() if c["state"] else None)
    return out


def _plain_norm(s):
    c, x, res, wt = s["case"], s["x"].float(), s["residual"], s["weight"]
    hs = None if res is None else (x + res.float()).to(res.dtype)
    h = x if hs is None else hs.float()
    rstd = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
    y = h * rstd * wt
    if c["do"] == "fp8":
        M, D = y.shape
        g = D if c["group"] == 0 else c["group"]
        n = -(-D // g)
        yp = torch.cat((y, y.new_zeros(M, n * g - D)), 1).view(M, n, g)
        scales = torch.clamp(yp.abs().amax(2), min=AMAX_FLOOR) / E4M3_MAX
        q = torch.clamp(yp / scales[..., None], -E4M3_MAX, E4M3_MAX).view(M, n * g)[:, :D]
        return dict(q=q.to(torch.float8_e4m3fn), scales=scales, h=hs)
    out = dict(y=y.to(torch.bfloat16), h=hs)
    if c["do"] == "train":
        dy = s["dy"].float()
        n, t = h * rstd, wt * dy
        dh = rstd * (t - n * (t * n).mean(1, keepdim=True))
        if s["dh"] is not None:
            dh = dh + s["dh"].float()
        out.update(dx=dh.to(torch.bfloat16), dresidual=dh if c["res"] == "fp32" else None,
                   dweight=(dy * n).sum(0, dtype=torch.float64).float())
    return out


# ------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(s) if case["op"] == "norm" else _exact_recurrence(s)


def _exact_recurrence(s):
    """Token after token from the definition; gradients by differentiating that."""
    c = s["case"]
    train = c["do"] == "train"
    f = {k: s[k].double().requires_grad_(train) for k in ("x1", "x2", "x3", "gate", "log_rate", "Dskip", "state_in",
                                                          "state") if s.get(k) is not None}
    log_a = f["log_rate"] * torch.sigmoid(f["gate"])
    a, w = log_a.exp(), (-torch.expm1(2 * log_a)).sqrt() if c["normalize"] else 1.0
    if s.get("reset") is not None:
        r = s["reset"].bool()[..., None]
        a = a.masked_fill(r, 0.0)
        w = w.masked_fill(r, 1.0) if c["normalize"] else w
    v = f["x1"] * f["x2"]
    u = w * v
    skip = f["Dskip"] * v if "Dskip" in f else 0.0
    if c["do"] == "decode":
        st = a * f["state"] + u
        return dict(y=f["x3"] * st + skip, state=st)
    h = f["state_in"] if "state_in" in f else torch.zeros_like(u[:, 0])
    states = []
    for at, ut in zip(a.unbind(1), u.unbind(1)):
        h = torch.addcmul(ut, at, h)
        states.append(h)
    y = f["x3"] * torch.stack(states, 1) + skip
    out = dict(y=y.detach(), state_out=h.detach())
    if train:
        loss = (y * s["dy"].double()).sum()
        if s["dstate_out"] is not None:
            loss = loss + (h * s["dstate_out"].double()).sum()
        loss.backward()
        out.update({"d" + k: f[k].grad for k in ("x1", "x2", "x3", "gate", "log_rate", "Dskip", "state_in") if k in f})
    return out


def _exact_norm(s):
    c, x, wt = s["case"], s["x"].double(), s["weight"].double()
    train = c["do"] == "train"
    h = x if s["residual"] is None else x + s["residual"].double()
    held = None if s["residual"] is None else h
    # the norm is taken of the stream as it is held
    h = h if s["residual"] is None else h.to(s["residual"].dtype).double()
    if train:
        h, wt = h.requires_grad_(), wt.requires_grad_()
    y = h * wt / (h.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
    if c["do"] == "fp8":
        g = y.shape[1] if c["group"] == 0 else c["group"]
        parts = y.abs().split(g, 1)
        scales = torch.stack([p.max(1).values for p in parts], 1) / E4M3_MAX
        q = torch.cat([p / scales[:, i:i + 1] for i, p in enumerate(y.split(g, 1))], 1)
        return dict(q=q, scales=scales, h=held)
    out = dict(y=y.detach(), h=held)
    if train:
        loss = (y * s["dy"].double()).sum()
        if s["dh"] is not None:
            loss = loss + (h * s["dh"].double()).sum()
        loss.backward()
        out.update(dx=h.grad, dresidual=h.grad if c["res"] == "fp32" else None, dweight=wt.grad)
    return out
