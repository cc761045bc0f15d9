"""Pins of the oracle's layers: forward passes against torch's in binary64,
gradients against torch's and against central differences, block codes against
``int8.quantize`` of each block and against rational arithmetic."""

import numpy as np
import pytest
import torch

from oracle import int8 as o8, layers as ol


def _central(f, x, along, h=1e-5):
    return (f(x + h * along) - f(x - h * along)) / (2 * h)


@pytest.mark.parametrize("cols", [1, 5, 128, 130, 300])
@pytest.mark.parametrize("rounding", ["rn", "sr"])
def test_block_codes_are_row_codes_of_the_blocks(cols, rounding):
    rng = np.random.default_rng(cols)
    x = (rng.standard_normal((4, cols)) * 10.0 ** rng.integers(-3, 3, (4, 1))).astype(np.float32)
    x[1, 0] = np.inf
    x[2] = 0.0
    q, s = ol.pack(x, rounding, 3, 5, 17)
    for r in range(4):
        for b, c in enumerate(range(0, cols, ol.BLOCK)):
            want, scale = o8.quantize(x[r:r + 1, c:c + ol.BLOCK], False, rounding, 3, 5,
                                      17 + r * cols + c)
            assert np.array_equal(q[r:r + 1, c:c + ol.BLOCK], want)
            assert np.array_equal(s[r, b:b + 1], scale, equal_nan=True)
    assert np.isnan(s[1, 0]) and not q[2].any() and not s[2].any()


def test_block_codes_of_binary64_values():
    """Values that binary32 would move over a border between two codes."""
    s = np.float64(np.float32(1.0 / 127.0))
    x = np.zeros((1, 128))
    x[0, 0] = 1.0
    x[0, 1] = 3.5 * s * (1 + 1e-12)
    x[0, 2] = 3.5 * s * (1 - 1e-12)
    x[0, 3] = -x[0, 2]
    q, _ = ol.pack(x)
    assert q[0, :4].tolist() == [127, 4, 3, -3]


@pytest.mark.parametrize("params", ["wb", "w", "b", ""])
def test_layer_norm(params):
    rng = np.random.default_rng(len(params))
    x, dy = rng.standard_normal((2, 7, 33)) + 0.5
    w = rng.standard_normal(33) if "w" in params else None
    b = rng.standard_normal(33) if "b" in params else None
    y, xh, rstd = ol.layer_norm(x, w, b, 1e-3)
    dx, dw, db = ol.layer_norm_grads(dy, xh, rstd, w)
    leaves = [None if v is None else torch.tensor(v, requires_grad=True) for v in (x, w, b)]
    want = torch.nn.functional.layer_norm(leaves[0], (33,), leaves[1], leaves[2], 1e-3)
    want.backward(torch.tensor(dy))
    assert np.allclose(y, want.detach().numpy(), rtol=1e-12, atol=1e-12)
    for got, leaf in zip((dx, dw, db), leaves):
        if leaf is not None:
            assert np.allclose(got, leaf.grad.numpy(), rtol=1e-10, atol=1e-12)
    along = rng.standard_normal(x.shape)
    change = _central(lambda v: np.sum(dy * ol.layer_norm(v, w, b, 1e-3)[0]), x, along)
    assert abs(change - np.sum(dx * along)) < 1e-7 * np.sum(np.abs(dx * along))


def test_silu_mul():
    rng = np.random.default_rng(2)
    gate, up, dy = rng.standard_normal((3, 6, 40)) * 3
    g, u = torch.tensor(gate, requires_grad=True), torch.tensor(up, requires_grad=True)
    y = torch.nn.functional.silu(g) * u
    y.backward(torch.tensor(dy))
    assert np.allclose(ol.silu_mul(gate, up), y.detach().numpy(), rtol=1e-12)
    dgate, dup = ol.silu_mul_grads(dy, gate, up)
    assert np.allclose(dgate, g.grad.numpy(), rtol=1e-10, atol=1e-14)
    assert np.allclose(dup, u.grad.numpy(), rtol=1e-10, atol=1e-14)
    along = rng.standard_normal(gate.shape)
    change = _central(lambda v: np.sum(dy * ol.silu_mul(v, up)), gate, along)
    assert abs(change - np.sum(dgate * along)) < 1e-7 * np.sum(np.abs(dgate * along))


def test_embedding():
    rng = np.random.default_rng(3)
    w, ids = rng.standard_normal((11, 5)), np.array([3, 0, 3, 10, -1, 11, 3, 2])
    y = ol.embedding(ids, w, 2.5)
    assert np.array_equal(y[[0, 1, 3]], w[[3, 0, 10]] * 2.5) and np.isnan(y[[4, 5]]).all()
    dy = rng.standard_normal((8, 5))
    for padding in (None, 3):
        grad, size, count = ol.embedding_grad(ids, dy, 11, 2.5, padding)
        want = torch.tensor(w, requires_grad=True)
        ok = [0, 1, 2, 3, 6, 7]
        out = torch.nn.functional.embedding(torch.tensor(ids[ok]), want, padding_idx=padding) * 2.5
        out.backward(torch.tensor(dy[ok]))
        assert np.allclose(grad, want.grad.numpy(), rtol=1e-12, atol=1e-14)
        assert count.tolist() == [1, 0, 1, 3 if padding is None else 0] + [0] * 6 + [1]
        assert np.all(size >= np.abs(grad) - 1e-12)
