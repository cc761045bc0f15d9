"""The layers at the ends of their types' range: rows whose mean is far larger than
any spread, differences that overflow, sigmoids next to zero, long sums.

u = 2**-24, half a step of binary32."""

import numpy as np
import pytest
import torch

from oracle import layers as ol
from adamw_optimizer_stochastic_amd import embedding, layer_norm, silu_mul
from _gpu_util import announce, gpu, require_gpu
from test_gpu_layers import DTYPES, U, _check_norm, _close, _norm_codes, _np, _values

pytestmark = gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [1, 5, 100, 515, 1100, 2050, 4095, 8190, 9001, 24570])
def test_gradients_of_rows_of_one_large_value(cols, dtype):
    """mean * rstd overflows (rstd is 316 where var is 0): nothing past a row's end may
    come into its sums."""
    announce("norm of one large value", cols, dtype)
    rng = np.random.default_rng(cols)
    x = torch.tensor([1e38, -3e38, 2e36, -1.0, 0.0]).to(DTYPES[dtype])[:, None].expand(5, cols).contiguous().cuda()
    w, w64 = _values(rng, (cols,), torch.float32)
    dy, dy64 = _values(rng, (5, cols), DTYPES[dtype])
    for saved in ("input", "i8"):
        leaf, weight = x.clone().requires_grad_(), w.clone().requires_grad_()
        y = layer_norm(leaf, weight, saved=saved)
        dx, dw = torch.autograd.grad(y, [leaf, weight], dy)
        used = None
        if saved == "i8":
            used = ol.unpack(*ol.pack(ol.layer_norm(_np(x))[1])).astype(np.float64)
        _check_norm(_np(x), dy64, w64, None, 1e-5, y, dx, dw, None, used)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [128, 1000, 3001, 8192, 9001])
def test_codes_of_rows_whose_differences_overflow(cols, dtype):
    """x - mean past binary32's range, and rstd below its normal numbers: the codes are
    those of the 64-bit normalised rows all the same."""
    announce("norm codes of overflowing differences", cols, dtype)
    rng = np.random.default_rng(cols + 7)
    x = np.empty((6, cols))
    x[0] = 2e38 * rng.uniform(0.9, 1.1, cols)
    x[0, 3] = -3.2e38
    x[1] = -x[0]
    x[2] = rng.choice([-3.3e38, 3.3e38], cols)
    x[3] = rng.uniform(-3e38, 3e38, cols)
    x[4] = np.where(rng.random(cols) < 0.9, 3.3e38, rng.uniform(-3.3e38, 3.3e38, cols))
    x[5] = rng.uniform(-9e37, 9e37, cols)
    t = torch.from_numpy(x.astype(np.float32)).to(DTYPES[dtype]).cuda()
    q, s = _norm_codes(t, None, None, 1e-5)
    want_q, want_s = ol.pack(ol.layer_norm(_np(t))[1])
    assert np.array_equal(s.cpu().numpy(), want_s)
    assert np.array_equal(q.cpu().numpy()[:, :cols], want_q)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("saved", ["inputs", "i8"])
def test_silu_gradient_whose_factors_overflow_together(saved, dtype):
    """dy * up past binary32's range where the gradient is not: the sigmoid's factor is
    there before both of them are. Powers of two, alone in their blocks of codes (whose
    rounding is up's alone: half a step of 1/127)."""
    announce("silu_mul of large factors", saved, dtype)
    gate = torch.tensor([-40.0, -20.0, -10.0, 4.0, 30.0])[:, None].to(DTYPES[dtype]).cuda()
    up, dy = (torch.full_like(gate, 2.0 ** e) for e in (70, 62))
    dy[3:] = 2.0 ** 50
    leaves = [gate.requires_grad_(), up.requires_grad_()]
    dgate, dup = torch.autograd.grad(silu_mul(*leaves, saved=saved), leaves, dy)
    want_g, want_u = ol.silu_mul_grads(_np(dy), _np(gate), _np(up))
    # sigmoids: in bf16 off by (|gate| + 6) 2**-22 of themselves, 46 * 2**-22 at most, in f32
    # by the functions' 4 u; a gate that its code (127) stands for is off by 2**-23 of
    # itself, which moves them by 40 * 2**-23. Products 8 u, and half a step of the result.
    off = 66 * 2.0 ** -22 + 8 * U + (2.0 ** -8 if dtype == "bf16" else 0.0)
    assert np.all(np.isfinite(want_g)) and np.all(np.abs(want_g) < 3e38)
    assert np.all(np.abs(_np(dgate) - want_g) <= off * np.abs(want_g))
    assert np.all(np.abs(_np(dup) - want_u) <= off * np.abs(want_u))


# Values whose f32 sums in one chain of additions drift most: n of each in a row are off by
# n / 4 half steps, one way.
DRIFT = np.float32([1.9988405, 1.0041199, 1.8167114, 1.02771, 1.992431, 1.9191899, 1.9130845, 1.9775362])


@pytest.mark.parametrize("saved", ["input", "i8"])
@pytest.mark.parametrize("rows,cols,groups", [(2 ** 24 - 1, 4, 16), (2 ** 20 - 3, 4100, 1), (2 ** 20 - 3, 8200, 1)])
def test_parameter_gradients_of_many_rows(rows, cols, groups, saved):
    """Equal rows and one gradient a column: a lane's sum of t = rows / 256 / groups rows is
    256 and t / 256 additions in a row, the groups and 256 workgroups 16 and 68 more, a
    term 7 operations."""
    announce("norm gradients of many rows", rows, cols, saved)
    rng = np.random.default_rng([rows, cols])
    row, row64 = _values(rng, (1, cols), torch.float32, 2.0)
    c = np.resize(DRIFT, cols)
    x = row.expand(rows, cols).contiguous()
    dy = torch.from_numpy(c).cuda()[None].expand(rows, cols).contiguous()
    w, b = (torch.ones(cols, device="cuda", requires_grad=True) for _ in range(2))
    dw, db = torch.autograd.grad(layer_norm(x, w, b, saved=saved), [w, b], dy)
    h = ol.layer_norm(row64)[1][0]
    if saved == "i8":
        h = ol.unpack(*ol.pack(h[None])).astype(np.float64)[0]
    t = -(-rows // (256 * groups))
    chain = 256 + -(-t // 256) + 16 + 68
    _close(db, rows * c.astype(np.float64), chain * U * rows * c, "db")
    _close(dw, rows * c.astype(np.float64) * h, (chain + 7) * U * rows * c * np.abs(h), "dw")


def test_embedding_gradient_of_a_frequent_id():
    """2**24 tokens of one id: chunks of 16384 positions, each 256 + 64 additions in a row,
    1024 of them by 4 shares of 256."""
    announce("embedding gradient of a frequent id")
    n, dim = 2 ** 24, 8
    dy = torch.from_numpy(DRIFT).cuda()[None].expand(n, dim).contiguous()
    ids = torch.ones(n, dtype=torch.int32, device="cuda")
    w = torch.zeros(3, dim, device="cuda", requires_grad=True)
    dw, = torch.autograd.grad(embedding(ids, w), w, dy)
    want = n * DRIFT.astype(np.float64)
    assert not dw[0].any() and not dw[2].any()
    _close(dw[1], want, (256 + 64 + 256 + 4 + 2) * U * want, "dw")
