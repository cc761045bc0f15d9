"""Newton-Schulz orthogonalisation and the Muon step in binary64 (oracle side).

``newton_schulz`` is the definition. ``newton_schulz_f16`` makes the
roundings that f16 operands with X held as two f16 numbers bring, and none
else (sums and everything between two roundings in binary64): how far it
is from the definition on an input says what accuracy that scheme has
there, apart from any kernel. Both take and give torch float64 matrices, on
any device.

Test infrastructure only (see the package header).
"""

import math

import torch

COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def newton_schulz(g, steps=5, coefficients=COEFFICIENTS, eps=1e-7):
    a, b, c = coefficients
    x = g.double()
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    x = x / (torch.sqrt((x * x).sum()) + eps)
    for _ in range(steps):
        gram = x @ x.T
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.T if tall else x


def _f16(x, scale):
    return (x * scale).to(torch.float16).double() / scale


def newton_schulz_f16(g, steps=5, coefficients=COEFFICIENTS, eps=1e-7):
    a, b, c = coefficients
    x = g.double()
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    s, t = x.shape
    sx = 2.0 ** min(14, round(math.log2(math.sqrt(s * t))))
    sa = 2.0 ** min(14, round(math.log2(s)))
    x = x / (torch.sqrt((x * x).sum()) + eps)
    for k in range(steps):
        hi = _f16(x, sx)
        lo = _f16(x - hi, sx)
        gram = _f16(hi @ hi.T, sa)
        poly = _f16(b * gram + c * (gram @ gram), sa)
        x = a * (hi + lo) + poly @ hi
    return x.T if tall else x


def relative(x, y):
    """|x - y| / |y| in the Frobenius norm (0 / 0 = 0)."""
    d, n = torch.linalg.norm(x.double() - y.double()).item(), torch.linalg.norm(y.double()).item()
    return d / n if n else (math.inf if d else 0.0)
