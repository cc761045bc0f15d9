"""Pins of oracle/int8.py: its codes against rational arithmetic, next to
every kind of border, and the sums against Python integers (CPU only)."""

import numpy as np
import pytest

import oracle
from oracle import int8 as o8


def _near_borders(s, rng, n=400):
    """binary32 values on, one step below and one step above (k + 1/2) s and k s."""
    k = rng.integers(0, 127, n)
    half = rng.integers(0, 2, n) * 0.5
    v = ((k + half) * float(s)).astype(np.float32)
    return np.concatenate([v, np.nextafter(v, np.float32(0)), np.nextafter(v, np.float32(1e30)), -v])


@pytest.mark.parametrize("amax", [127.0, 1.0, 3.7e-3, 1e30, 2.0 ** -119, 0.9999999])
def test_codes_match_rational_arithmetic(amax):
    rng = np.random.default_rng(int(amax * 1000) % 2 ** 31)
    s = o8.scale_of(np.float32(amax))
    x = np.concatenate([[np.float32(amax)], _near_borders(s, rng),
                        (rng.standard_normal(300) * amax / 3).astype(np.float32)])
    x = np.clip(x, -np.float32(amax), np.float32(amax))[None, :]
    q, got = o8.quantize(x)
    assert got[0] == s
    assert [int(v) for v in q[0]] == [o8.code_scalar(v, s) for v in x[0]]
    q, _ = o8.quantize(x, rounding="sr", seed=5, step=9, base_index=3)
    r = oracle.random16(np.arange(3, 3 + x.size, dtype=np.uint64), 5, 9)
    assert [int(v) for v in q[0]] == [o8.code_scalar(v, s, b) for v, b in zip(x[0], r)]


def test_scale_is_the_nearest_binary32():
    from fractions import Fraction
    rng = np.random.default_rng(1)
    for a in (rng.standard_normal(2000) * 10.0 ** rng.integers(-30, 30, 2000)).astype(np.float32):
        a = abs(a)
        s = o8.scale_of(a)
        t = Fraction(float(a)) / 127
        err = abs(Fraction(float(s)) - t)
        for n in (np.nextafter(s, np.float32(0)), np.nextafter(s, np.float32(np.inf))):
            assert err <= abs(Fraction(float(n)) - t)


def test_groups_that_are_empty_tiny_or_not_finite():
    x = np.array([[0, 0, 0], [1e-40, -2e-38, 0], [1, np.inf, 2], [np.nan, 1, 2], [1, 2, -4]],
                 np.float32)
    q, s = o8.quantize(x)
    assert s[0] == 0 and s[1] == 0 and np.isnan(s[2]) and np.isnan(s[3]) and s[4] > 0
    assert not q[:4].any() and list(q[4]) == [32, 64, -127]
    qt, st = o8.quantize(x.T, transpose=True)
    assert np.array_equal(qt, q) and np.array_equal(st, s, equal_nan=True)
    q, s = o8.quantize(np.zeros((0, 4), np.float32), transpose=True)
    assert q.shape == (4, 0) and not s.any()


def test_transposed_codes_take_the_bits_of_the_same_elements():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 7)).astype(np.float32)
    x[0, :] = x[:, 0] = 0
    x[0, 0] = 9          # one maximum for every row and column that has it
    a, _ = o8.quantize(np.full((5, 7), 1.0, np.float32) * x, rounding="sr", seed=1, step=2)
    b, _ = o8.quantize(x, transpose=True, rounding="sr", seed=1, step=2)
    same = o8.quantize(x[:1], rounding="sr", seed=1, step=2)[0]
    assert np.array_equal(a[:1], same) and b.shape == (7, 5)
    # stochastic codes are one of the two neighbours
    for q, y in ((a, x), (b, x.T)):
        s = o8.scale_of(np.abs(y).max(1)).astype(np.float64)[:, None]
        t = np.abs(y) / np.where(s == 0, 1, s)
        assert np.all((np.abs(q) == np.floor(t)) | (np.abs(q) == np.ceil(t)))


def test_product_sums_are_exact():
    rng = np.random.default_rng(3)
    a = rng.integers(-128, 128, (3, 5000)).astype(np.int8)
    b = rng.integers(-128, 128, (4, 5000)).astype(np.int8)
    got = o8.gemm_f32(a, b, np.ones(3, np.float32), np.ones(4, np.float32))
    want = [[np.float32(sum(int(x) * int(y) for x, y in zip(r, c))) for c in b] for r in a]
    assert np.array_equal(got, np.array(want, np.float32))
