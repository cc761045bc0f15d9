"""Ceilings on the error of the Newton-Schulz products, by class of matrix, and
special matrices on the path of many workgroups.

The other tests hold the kernel to the error that its scheme of roundings has
on the same input; these hold the scheme itself to what is documented. O is
taken unrounded: a Muon step on f32 zeros with lr 1, no momentum and no decay
leaves -O. The ceilings: the scheme in binary64 (oracle.muon.newton_schulz_f16)
on some 40,000 matrices of 1 to 200 by 1 to 4099 was off by at most

  2.4e-3  varied entries (Gaussian, uniform, low rank, rank one, strong
          directions over a floor), short side 64 and more;
  3.2e-3  the same, short side 16 to 63;
  1.4e-2  few or equal roundings, which do not average: short sides of 1 to 15,
          entries of one magnitude (ones, signs of rank one or two), orthogonal
          rows, a single entry.

The kernel's roundings are the same in number and size and fall differently
only where f32 sums differ, so a quarter more than these covers its draws;
one singular value alone cannot be off by more than 4.5e-2."""

import pytest
import torch

from oracle import muon as om
from adamw_optimizer_stochastic_amd import ops
from _gpu_util import gpu, require_gpu, announce

pytestmark = gpu

VARIED, VARIED_SHORT, FEW = 3.0e-3, 4.0e-3, 1.75e-2
BF16 = 2.0 ** -8   # a bf16 rounding, of every value and so of the norm


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _matrix(kind, rows, cols, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + rows * 131 + cols)

    def n(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    r = max(1, min(rows, cols) // 16)
    if kind == "normal":
        return n(rows, cols)
    if kind == "uniform":
        return torch.rand((rows, cols), generator=gen, device="cuda")
    if kind == "lowrank":
        return n(rows, r) @ n(r, cols)
    if kind == "rank1":
        return n(rows, 1) * n(1, cols)
    if kind == "floor":
        return n(rows, r) @ n(r, cols) / r ** 0.5 + 0.1 * n(rows, cols)
    if kind == "ones":
        return torch.ones(rows, cols, device="cuda")
    if kind == "sign1":
        return torch.sign(n(rows, 1)) * torch.sign(n(1, cols))
    if kind == "sign2":
        return (torch.sign(n(rows, 1)) * torch.sign(n(1, cols))
                + 0.5 * torch.sign(n(rows, 1)) * torch.sign(n(1, cols)))
    if kind == "eye":
        return torch.eye(rows, cols, device="cuda")
    assert kind == "one"
    x = torch.zeros(rows, cols, device="cuda")
    x[rows // 2, cols // 2] = -5.0
    return x


def _unrounded(g):
    p, m = torch.zeros_like(g), torch.zeros_like(g)
    ops.muon_step([p], [g], [m], [0], lr=1.0, momentum=0.0, nesterov=False, adjust_lr="original",
                  step=1, seed=0)
    return -p / ops.muon_lr_factor(*g.shape)


def _hold(kind, shape, ceiling):
    announce("newton_schulz ceiling", kind, shape)
    for seed in range(3):
        for s in {shape, shape[::-1]}:
            g = _matrix(kind, *s, seed)
            want = om.newton_schulz(g)
            # (dividing by the shape's factor costs two binary32 roundings)
            assert om.relative(_unrounded(g), want) <= ceiling + 2.0 ** -22, (s, seed)
            assert om.relative(ops.newton_schulz(g), want) <= ceiling + BF16, (s, seed)


@pytest.mark.parametrize("kind", ["normal", "uniform", "lowrank", "rank1", "floor"])
@pytest.mark.parametrize("shape", [(64, 64), (64, 700), (100, 130), (128, 128), (200, 333), (260, 2000),
                                   (700, 700), (1024, 1100)])
def test_varied(kind, shape):
    _hold(kind, shape, VARIED)


@pytest.mark.parametrize("kind", ["normal", "uniform", "lowrank", "rank1", "floor"])
@pytest.mark.parametrize("shape", [(16, 16), (16, 130), (17, 2000), (31, 700), (32, 2000), (48, 100), (63, 64)])
def test_varied_with_a_short_side(kind, shape):
    _hold(kind, shape, VARIED_SHORT)


@pytest.mark.parametrize("kind", ["normal", "uniform", "floor", "ones", "sign1"])
@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (1, 4099), (2, 3), (2, 300), (3, 100), (3, 4096), (4, 256),
                                   (5, 2000), (8, 300), (12, 700)])
def test_few_rows(kind, shape):
    _hold(kind, shape, FEW)


@pytest.mark.parametrize("kind", ["ones", "sign1", "sign2", "eye", "one"])
@pytest.mark.parametrize("shape", [(16, 700), (59, 125), (64, 64), (130, 700), (150, 200), (300, 500)])
def test_equal_entries(kind, shape):
    _hold(kind, shape, FEW)


LARGE = [(200, 333), (333, 200), (64, 1030), (700, 130)]


def _same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", LARGE)
def test_bad_matrices_beside_good_ones(shape, dtype):
    """Zeros, one Inf or NaN (also in the last row and column) and a good matrix in
    one launch: zeros give zeros, NaN and Inf only NaN, and the others are as
    alone."""
    announce("newton_schulz special, large", shape, dtype)
    assert ops.muon_workspace_bytes([shape]) > 0   # (not the one-workgroup kernel)
    rows, cols = shape
    good = _matrix("floor", rows, cols, 1).to(dtype)
    alone = ops.newton_schulz(good)
    for value in (float("nan"), float("inf"), float("-inf")):
        for i, j in ((0, 0), (rows - 1, cols - 1), (rows // 2, 3)):
            bad = good.clone()
            bad[i, j] = value
            o = ops.newton_schulz(torch.stack([good, torch.zeros_like(good), bad, good]))
            torch.cuda.synchronize()
            assert _same(o[0], alone) and _same(o[3], alone)
            assert not bool(o[1].any())
            assert bool(torch.isnan(o[2]).all())


@pytest.mark.parametrize("shape", LARGE)
def test_extreme_norms(shape):
    """Huge and tiny values, with and without an eps beside the norm, a single
    entry, and an eps next to the norm."""
    announce("newton_schulz extreme, large", shape)
    for scale in (1e38, 1e-30):
        g = _matrix("normal", *shape, 2).clamp(-3, 3) * scale
        want = om.newton_schulz(g, eps=0.0)
        assert om.relative(ops.newton_schulz(g, eps=0.0), want) <= VARIED + BF16, scale
    one = _matrix("one", *shape, 0)
    assert om.relative(ops.newton_schulz(one), om.newton_schulz(one)) <= FEW + BF16
    small = torch.full(shape, 1e-10, device="cuda")
    want = om.newton_schulz(small)
    assert om.relative(ops.newton_schulz(small), want) <= FEW + BF16


@pytest.mark.parametrize("shape", LARGE + [(64, 64)])
def test_step_with_a_bad_gradient(shape):
    """A NaN in one gradient: all of that matrix is NaN, its momentum in that
    element; the matrix beside it moves as alone."""
    announce("muon_step bad gradient", shape)
    start = _matrix("normal", *shape, 3).bfloat16()
    good = _matrix("floor", *shape, 4).bfloat16()
    bad = good.clone()
    bad[shape[0] - 1, shape[1] - 1] = float("nan")
    zeros = torch.zeros(shape, device="cuda")
    p, m = start.clone(), zeros.clone()
    ops.muon_step([p], [good], [m], [7], lr=0.02, weight_decay=0.1, step=1, seed=3)
    ps, ms = [start.clone(), start.clone()], [zeros.clone(), zeros.clone()]
    ops.muon_step(ps, [bad, good], ms, [0, 7], lr=0.02, weight_decay=0.1, step=1, seed=3)
    torch.cuda.synchronize()
    assert _same(ps[1], p) and torch.equal(ms[1], m)
    assert bool(torch.isnan(ps[0]).all())
    assert torch.equal(torch.isnan(ms[0]), torch.isnan(bad))


@pytest.mark.parametrize("shape", [(1, 7), (64, 64)] + LARGE)
def test_norm_far_below_eps(shape):
    """X below f16's range: each of its elements is off by at most half of f16's
    smallest number over X's scale, 2**-25 / sx with sx > sqrt(s t) / 2, so X by
    2**-24 in the Frobenius norm, a step, and the result by 2**-24 * (3.4445**5 +
    .. + 3.4445) = 2**-24 * 682 = 4.1e-5 (B X adds less than 5 X**3 = 1e-9 a step: X is
    below 5e-4 throughout)."""
    announce("newton_schulz below eps", shape)
    for scale in (1e-13, 1e-14, 1e-16):
        g = _matrix("normal", *shape, 5)
        g = g / torch.linalg.norm(g) * scale
        want = om.newton_schulz(g)
        d = torch.linalg.norm(ops.newton_schulz(g).double() - want).item()
        assert d <= 4.1e-5 + BF16 * torch.linalg.norm(want).item()
