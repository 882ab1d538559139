"""The e4m3 codes of the norm are those of the fp32 quotient y / scale.

Rows of +-1 with eps = 0 have a mean square and rstd of 1 exactly, so that y is
the weight, bit for bit, and the scale and the codes follow from it: scale =
max|w| / 448 in fp32 and the e4m3 value nearest to the fp32 quotient w / scale
(ties to even).  The weights put that quotient on the borders between two codes
and next to them, where any other way to form it shows.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def borders():
    """Values half-way between neighbouring e4m3 codes, below 448: 8.5 .. 14.5
    times a power of two, and of the subnormals' steps of 2^-9."""
    z = [(m + 0.5) * 2.0 ** e for e in range(-9, 6) for m in range(8, 16) if (m + 0.5) * 2.0 ** e < 448]
    return np.array(z + [(k + 0.5) * 2.0 ** -9 for k in range(8)], dtype=np.float64)


def weights(rng, n, amax):
    """n weights with the largest |w| = amax at a random place, the others a
    border times the scale, or that value's fp32 neighbours."""
    scale = np.float32(amax) / np.float32(448)
    w = (rng.choice(borders(), n) * np.float64(scale)).astype(np.float32)
    w = np.nextafter(w, w * np.float32(2) * rng.integers(0, 2, n).astype(np.float32)) if rng.random() < 0.5 else w
    w *= rng.choice(np.array([-1, 1], np.float32), n)
    w[rng.integers(n)] = amax
    return w


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("res", [None, "bf16", "fp32"])
@pytest.mark.parametrize("D", [8, 64, 136, 256, 1000, 4096, 16384])
def test_codes_are_the_quotients(D, res, group):
    import torch
    import hyena_long_convolution_b200 as hy
    rng = np.random.default_rng(D + group)
    step = D if group == 0 else group
    for power in (0, 0, 0, 0, -70, -94, 90):
        w = np.concatenate([weights(rng, min(step, D - i), np.float32(rng.uniform(0.1, 9.0) * 2.0 ** power))
                            for i in range(0, D, step)])
        w = torch.from_numpy(w)
        x = torch.from_numpy(rng.choice([-1.0, 1.0], (3, D))).to(torch.bfloat16)
        r = None if res is None else torch.zeros(3, D, dtype=torch.bfloat16 if res == "bf16" else torch.float32)
        q, s = hy.rms_norm_fp8(x.cuda(), w.cuda(), 0.0, residual=None if r is None else r.cuda(), group=group)
        parts = w.split(step)
        scale = torch.stack([p.abs().max() / 448.0 for p in parts])
        want = torch.cat([p / c for p, c in zip(parts, scale)]) * x.float()
        assert torch.equal(s.cpu(), scale.expand(3, -1))
        assert torch.equal(q.cpu().float(), want.to(torch.float8_e4m3fn).float())
