"""Pins of oracle/muon.py (CPU only): the definition against singular values
mapped one by one, and the accuracy that f16 operands with X in two parts have
on matrices that a coarser scheme loses."""

import numpy as np
import pytest
import torch

from oracle import muon as om


def _matrix(kind, m, n, seed=0):
    rng = np.random.default_rng([seed, m, n])
    if kind == "normal":
        x = rng.standard_normal((m, n))
    elif kind == "decay":
        u = np.linalg.qr(rng.standard_normal((m, min(m, n))))[0]
        v = np.linalg.qr(rng.standard_normal((n, min(m, n))))[0]
        x = (u * np.logspace(0, -3, min(m, n))) @ v.T
    else:
        r = max(1, min(m, n) // 16)
        x = rng.standard_normal((m, r)) @ rng.standard_normal((r, n))
    return torch.from_numpy(x).bfloat16().double()


@pytest.mark.parametrize("shape", [(5, 5), (7, 30), (30, 7), (1, 9)])
def test_definition_maps_singular_values(shape):
    """Newton-Schulz applies x -> a x + b x^3 + c x^5 to every singular value and
    leaves the singular vectors."""
    g = _matrix("normal", *shape)
    u, s, vt = np.linalg.svd(g.numpy(), full_matrices=False)
    s = s / (np.sqrt((s ** 2).sum()) + 1e-7)
    a, b, c = om.COEFFICIENTS
    for _ in range(5):
        s = a * s + b * s ** 3 + c * s ** 5
    assert om.relative(om.newton_schulz(g), torch.from_numpy((u * s) @ vt)) < 1e-12


@pytest.mark.parametrize("kind", ["normal", "decay", "lowrank"])
@pytest.mark.parametrize("shape", [(64, 64), (48, 200), (200, 48), (1, 50), (256, 300)])
def test_two_part_f16_accuracy(kind, shape):
    """Within the rounding of the bf16 result (2**-8 of each value), where the
    roundings of many singular directions average. A matrix of one row has
    one direction: s -> s (a + B), B = b A + c A^2, A = s^2. With |B| <= 2.81
    and |b A + 2 c A^2| <= 1.55 on s in [0.7, 1.2], the roundings of A (its two
    operands' among them), of B and of the operand beside B move one step by at
    most 1.2 (3 * 1.55 + 2 * 2.81) 2**-11 = 6e-3. From s = 1 the orbit is 0.701, 1.114,
    0.721, 1.089, 0.70 with slopes -1.142, 1.31, -1.257, 0.745 behind its first
    four steps, so the five steps' errors add up to at most 5.3 * 6e-3 =
    3.2e-2, of 0.70: 1/16 covers it to second order."""
    g = _matrix(kind, *shape)
    tol = 2.0 ** -4 if min(shape) == 1 else 2.0 ** -8
    assert om.relative(om.newton_schulz_f16(g), om.newton_schulz(g)) < tol


def test_zero_matrix():
    z = torch.zeros(4, 6, dtype=torch.float64)
    assert not om.newton_schulz(z).any() and not om.newton_schulz_f16(z).any()
