"""fp64 oracle of the gated linear recurrence and its gradient: plain numpy,
token after token, from the definition.  Test infrastructure only.

    l_t = log_rate sigmoid(gate_t);  a_t = exp(l_t), 0 where reset_t
    s_t = a_t s_{t-1} + w_t v_t,  v = x1 x2,  w_t = sqrt(1 - a_t^2) or 1
    y_t = x3_t s_t + Dskip v_t

All arrays are float64, [B, L, D]; log_rate and Dskip [D]; reset [B, L] bool;
states [B, D].  Each function also returns the same sums with every term's
absolute value, the scale that a rounding error is measured against.
"""
from __future__ import annotations

from typing import NamedTuple

import numpy as np


class Forward(NamedTuple):
    y: np.ndarray
    state_out: np.ndarray
    states: np.ndarray   # s_t
    scale: np.ndarray    # s_t with |u|, |state_in| in the place of u, state_in


class Gates(NamedTuple):
    sig: np.ndarray
    a: np.ndarray
    w: np.ndarray


def gates(gate, log_rate, normalize, reset=None) -> Gates:
    with np.errstate(over="ignore"):
        sig = 1.0 / (1.0 + np.exp(-gate))
    l = log_rate * sig
    a = np.exp(l)
    w = np.sqrt(-np.expm1(2.0 * l)) if normalize else np.ones_like(a)
    if reset is not None:
        a = np.where(reset[..., None], 0.0, a)
        w = np.where(reset[..., None], 1.0, w)
    return Gates(sig, a, w)


def forward(x1, x2, x3, gate, log_rate, Dskip=None, reset=None, normalize=True, state_in=None) -> Forward:
    B, L, D = x1.shape
    g = gates(gate, log_rate, normalize, reset)
    v = x1 * x2
    u = g.w * v
    s = np.zeros((B, D)) if state_in is None else state_in.astype(np.float64)
    m = np.abs(s)
    states, scale = np.empty((B, L, D)), np.empty((B, L, D))
    for t in range(L):
        if reset is not None:  # a reset passes nothing, not even a NaN
            s = np.where(reset[:, t, None], 0.0, s)
            m = np.where(reset[:, t, None], 0.0, m)
        s = g.a[:, t] * s + u[:, t]
        m = g.a[:, t] * m + np.abs(u[:, t])
        states[:, t], scale[:, t] = s, m
    y = x3 * states
    if Dskip is not None:
        y = y + Dskip * v
    return Forward(y, s, states, scale)


class Backward(NamedTuple):
    dx1: np.ndarray
    dx2: np.ndarray
    dx3: np.ndarray
    dgate: np.ndarray
    dlog_rate: np.ndarray
    dDskip: np.ndarray
    dstate_in: np.ndarray
    scales: dict         # by the names above


def backward(dy, x1, x2, x3, gate, log_rate, Dskip=None, reset=None, normalize=True, state_in=None,
             dstate_out=None) -> Backward:
    B, L, D = x1.shape
    g = gates(gate, log_rate, normalize, reset)
    f = forward(x1, x2, x3, gate, log_rate, Dskip, reset, normalize, state_in)
    v = x1 * x2
    e = np.zeros((B, D)) if dstate_out is None else dstate_out.astype(np.float64)
    m = np.abs(e)
    q, qm = np.empty((B, L, D)), np.empty((B, L, D))
    for t in range(L - 1, -1, -1):
        q[:, t] = x3[:, t] * dy[:, t] + e
        qm[:, t] = np.abs(x3[:, t] * dy[:, t]) + m
        e, m = g.a[:, t] * q[:, t], g.a[:, t] * qm[:, t]
        if reset is not None:
            e = np.where(reset[:, t, None], 0.0, e)
            m = np.where(reset[:, t, None], 0.0, m)
    first = np.zeros((B, 1, D)) if state_in is None else state_in[:, None]
    prev = np.concatenate([first, f.states[:, :-1]], 1)
    prevm = np.concatenate([np.abs(first), f.scale[:, :-1]], 1)
    if normalize:
        ratio = np.divide(g.a * v, g.w, out=np.zeros_like(v), where=g.w > 0)
    else:
        ratio = np.zeros_like(v)
    dl = g.a * q * (prev - ratio)
    dlm = g.a * qm * (prevm + np.abs(ratio))
    if reset is not None:
        dl, dlm = (np.where(reset[..., None], 0.0, z) for z in (dl, dlm))
    skip = 0.0 if Dskip is None else Dskip
    dv, dvm = g.w * q + skip * dy, g.w * qm + np.abs(skip * dy)
    slope = log_rate * g.sig * (1.0 - g.sig)
    scales = dict(dx1=dvm * np.abs(x2), dx2=dvm * np.abs(x1), dx3=np.abs(dy) * f.scale, dgate=dlm * np.abs(slope),
                  dlog_rate=(dlm * g.sig).sum((0, 1)), dDskip=np.abs(dy * v).sum((0, 1)), dstate_in=m)
    return Backward(dv * x2, dv * x1, dy * f.states, dl * slope, (dl * g.sig).sum((0, 1)), (dy * v).sum((0, 1)), e,
                    scales)
