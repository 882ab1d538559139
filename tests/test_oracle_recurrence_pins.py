"""What pins the fp64 oracle of the gated recurrence: the fixed-pole modal
filter where the gate is constant, sequences apart where a reset cuts them,
a state carried between chunks, and differences for the gradient."""
import numpy as np
import pytest

import oracle
from oracle import recurrence as orec
from synth.inputs import bf16_bits_to_f32, make_modal_inputs


def draw(B, L, D, seed, state=True, resets=0.0):
    r = np.random.default_rng(seed)
    x = [r.standard_normal((B, L, D)) for _ in range(3)]
    return dict(x1=x[0], x2=x[1], x3=x[2], gate=1.5 * r.standard_normal((B, L, D)),
                log_rate=-np.exp(r.uniform(np.log(1e-3), 0.0, D)), Dskip=r.standard_normal(D),
                reset=r.random((B, L)) < resets if resets else None,
                state_in=r.standard_normal((B, D)) if state else None)


def test_constant_gate_is_the_modal_filter():
    """gate = 0 gives sigmoid = 1/2: one mode with log-pole log_rate / 2, residue 1."""
    B, L, D = 2, 50, 8
    inp = make_modal_inputs(B, L, D, 1, seed=5)
    x = [bf16_bits_to_f32(inp[k]).astype(np.float64) for k in ("x1", "x2", "x3")]
    S = np.random.default_rng(1).standard_normal((B, D, 1)).astype(np.float32)
    a = inp["log_poles"]
    ref_y, ref_S = oracle.modal_recurrence(inp["x1"], inp["x2"], inp["x3"], a, np.ones_like(a), inp["Dskip"], S)
    f = orec.forward(*x, np.zeros((B, L, D)), 2.0 * a[:, 0].astype(np.float64), inp["Dskip"].astype(np.float64),
                     normalize=False, state_in=S[..., 0].astype(np.float64))
    np.testing.assert_allclose(f.y, ref_y, rtol=0, atol=1e-12 * np.abs(ref_y).max())
    np.testing.assert_allclose(f.state_out, ref_S[..., 0], rtol=1e-12)


def test_normalised_constant_input_keeps_unit_variance():
    """E s^2 = a^2 E s^2 + (1 - a^2) E v^2: white v of variance 1 gives s of variance 1."""
    d = draw(4, 4000, 16, 3, state=False)
    d["log_rate"] = np.full(16, -0.5)
    d["x1"] = np.ones_like(d["x1"])
    f = orec.forward(**d)
    assert abs(np.var(f.states[:, 200:]) - 1.0) < 0.05


@pytest.mark.parametrize("normalize", [True, False])
def test_reset_cuts_sequences_apart(normalize):
    d = draw(1, 40, 4, 7)
    reset = np.zeros((1, 40), bool)
    reset[0, 17] = True
    f = orec.forward(**{**d, "reset": reset}, normalize=normalize)
    part = {k: v[:, 17:] if k in ("x1", "x2", "x3", "gate") else v for k, v in d.items()}
    first = reset[:, 17:]
    g = orec.forward(**{**part, "reset": first, "state_in": np.full((1, 4), np.nan)}, normalize=normalize)
    assert np.array_equal(f.y[:, 17:], g.y)
    h = orec.forward(**{k: v[:, :17] if k in ("x1", "x2", "x3", "gate") else v for k, v in d.items()},
                     normalize=normalize)
    assert np.array_equal(f.y[:, :17], h.y)


def test_chunks_equal_the_single_pass():
    d = draw(2, 37, 8, 9)
    f = orec.forward(**d)
    s, ys = d["state_in"], []
    for t0 in range(0, 37, 10):
        part = {k: v[:, t0:t0 + 10] if k in ("x1", "x2", "x3", "gate") else v for k, v in d.items()}
        g = orec.forward(**{**part, "state_in": s})
        s = g.state_out
        ys.append(g.y)
    assert np.array_equal(np.concatenate(ys, 1), f.y) and np.array_equal(s, f.state_out)


@pytest.mark.parametrize("normalize,resets", [(True, 0.0), (False, 0.0), (True, 0.2), (False, 0.2)])
def test_gradient_against_differences(normalize, resets):
    B, L, D = 2, 9, 3
    d = draw(B, L, D, 11, resets=resets)
    r = np.random.default_rng(12)
    dy, ds = r.standard_normal((B, L, D)), r.standard_normal((B, D))

    def loss(**kw):
        f = orec.forward(**{**d, **kw}, normalize=normalize)
        return float((f.y * dy).sum() + (f.state_out * ds).sum())

    g = orec.backward(dy, **d, normalize=normalize, dstate_out=ds)
    h = 1e-6
    for name in ("x1", "x2", "x3", "gate", "log_rate", "Dskip", "state_in"):
        num = np.empty_like(d[name])
        for i in np.ndindex(d[name].shape):
            p, m = d[name].copy(), d[name].copy()
            p[i] += h
            m[i] -= h
            num[i] = (loss(**{name: p}) - loss(**{name: m})) / (2 * h)
        got = getattr(g, "d" + name)
        # central differences: h^2 of the third derivative, 2^-53 |loss| / h of rounding
        np.testing.assert_allclose(got, num, rtol=1e-5, atol=1e-6, err_msg=name)
