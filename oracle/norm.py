"""fp64 oracle of the root-mean-square norm and its gradient: plain numpy, from
the definition.  Test infrastructure only.  h [rows, D] is the residual stream
as it is held (already rounded to its type)."""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100


def rstd(h, eps):
    return 1.0 / np.sqrt((h * h).mean(1) + eps)


def forward(h, weight, eps):
    return h * rstd(h, eps)[:, None] * weight


def scales(y, group):
    """max |y| / 448 per row (group = 0) or per `group` channels."""
    D = y.shape[1]
    g = D if group == 0 else group
    cols = [np.abs(y[:, i:i + g]).max(1) for i in range(0, D, g)]
    return np.maximum(np.stack(cols, 1), AMAX_FLOOR) / E4M3_MAX


def backward(dy, h, weight, eps, dh_out=None):
    """(dh, dweight, scale of dh's rounding errors, of dweight's)."""
    r = rstd(h, eps)[:, None]
    n, t = h * r, weight * dy
    dh = r * (t - n * (t * n).mean(1, keepdims=True))
    scale = r * (np.abs(t) + np.abs(n) * np.abs(t * n).mean(1, keepdims=True))
    if dh_out is not None:
        dh = dh + dh_out
        scale = scale + np.abs(dh_out)
    return dh, (dy * n).sum(0), scale, np.abs(dy * n).sum(0)
