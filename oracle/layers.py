"""Layer norm, gated SiLU, embedding and activations in 8 bits (oracle side).

The definitions in binary64, and the gradients as formulas; the codes of a
block of columns are ``int8.quantize``'s of a row of its elements.
``tests/test_oracle_layers.py`` pins them: gradients against differences, the
forward passes against torch's in binary64.

Test infrastructure only (see the package header).
"""

import numpy as np

from .stream import random16

BLOCK = 128


def _split(x, fill=0):
    """(rows, blocks, 128) of a matrix, its last block filled up."""
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    out = np.full((rows, blocks * BLOCK), fill, x.dtype)
    out[:, :cols] = x
    return out.reshape(rows, blocks, BLOCK)


def pack(x, rounding="rn", seed=0, step=0, base_index=0):
    """(codes int8, scales f32) of a matrix of binary32 or binary64 values. A
    binary64 value's code is that of itself; the scale is a binary32 number."""
    x = np.asarray(x)
    rows, cols = x.shape
    b = _split(x.astype(np.float64))
    with np.errstate(invalid="ignore", over="ignore"):
        amax = np.max(np.where(np.isnan(b), np.inf, np.abs(b)), axis=2)
        s = (amax / 127.0).astype(np.float32)
    s = np.where(np.isfinite(s), np.where(s < np.float32(2.0 ** -126), np.float32(0), s),
                 np.float32(np.nan)).astype(np.float32)
    live = s > 0
    div = np.where(live, s, 1).astype(np.float64)[:, :, None]
    t = np.where(live[:, :, None], np.abs(np.where(np.isfinite(b), b, 0)) / div, 0.0)
    if rounding == "sr":
        pos = (np.uint64(int(base_index) & 0xFFFFFFFFFFFFFFFF)
               + np.arange(rows * cols, dtype=np.uint64)).reshape(rows, cols)
        q = np.floor(t + _split(random16(pos, seed, step).astype(np.float64)) / 65536.0)
    else:
        q = np.rint(t)
    q = np.where(live[:, :, None], np.minimum(q, 127.0), 0.0) * np.sign(np.where(np.isnan(b), 0, b))
    return q.reshape(rows, -1)[:, :cols].astype(np.int8), s


def unpack(q, s):
    """f32(q * s), the values the codes stand for."""
    wide = np.repeat(np.asarray(s, np.float32), BLOCK, axis=1)[:, :q.shape[1]]
    return q.astype(np.float32) * wide


def layer_norm(x, w=None, b=None, eps=1e-5):
    """(y, xh, rstd) in binary64."""
    x = np.asarray(x, np.float64)
    d = x - x.mean(1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        rstd = 1.0 / np.sqrt((d * d).mean(1, keepdims=True) + eps)
        xh = d * rstd
    y = xh
    if w is not None:
        y = y * np.asarray(w, np.float64)
    if b is not None:
        y = y + np.asarray(b, np.float64)
    return y, xh, rstd


def layer_norm_grads(dy, xh, rstd, w=None):
    """(dx, dw, db) from the normalised rows, or from what their codes stand for."""
    dy, xh = np.asarray(dy, np.float64), np.asarray(xh, np.float64)
    g = dy if w is None else dy * np.asarray(w, np.float64)
    dx = rstd * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-np.asarray(g, np.float64)))


def silu_mul(gate, up):
    gate = np.asarray(gate, np.float64)
    return gate * sigmoid(gate) * np.asarray(up, np.float64)


def silu_mul_grads(dy, gate, up):
    """(dgate, dup)."""
    dy, gate, up = (np.asarray(v, np.float64) for v in (dy, gate, up))
    sig = sigmoid(gate)
    return dy * up * sig * (1.0 + gate * (1.0 - sig)), dy * gate * sig


def embedding(ids, w, scale=1.0):
    """Rows of w times scale; an id outside the table gives NaN."""
    ids, w = np.asarray(ids).reshape(-1), np.asarray(w, np.float64)
    there = (ids >= 0) & (ids < w.shape[0])
    y = np.full((ids.size, w.shape[1]), np.nan)
    y[there] = w[ids[there]] * scale
    return y


def embedding_grad(ids, dy, vocab, scale=1.0, padding=None):
    """(gradient, sum of the magnitudes, tokens of each row)."""
    ids, dy = np.asarray(ids).reshape(-1), np.asarray(dy, np.float64)
    keep = (ids >= 0) & (ids < vocab)
    if padding is not None:
        keep &= ids != padding
    total, size = np.zeros((vocab, dy.shape[1])), np.zeros((vocab, dy.shape[1]))
    np.add.at(total, ids[keep], dy[keep])
    np.add.at(size, ids[keep], np.abs(dy[keep]))
    return total * scale, size * abs(scale), np.bincount(ids[keep], minlength=vocab)
