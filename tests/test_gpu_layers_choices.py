"""The kernels that large calls take, each against the definitions and bit for bit
against the small calls' kernels on slices; every turn of a workgroup that walks many
rows; what calls write around their outputs and workspaces.

Tolerances: those counted in test_gpu_layers and test_gpu_embedding (u = 2**-24)."""

import numpy as np
import pytest
import torch

from oracle import layers as ol
from adamw_optimizer_stochastic_amd import _abi, embedding, layer_norm, linear_i8, ops, silu_mul
from _gpu_util import announce, gpu, require_gpu, to_host
from test_gpu_embedding import _check, _check_grad
from test_gpu_layers import (DTYPES, _check_norm, _close, _esig, _norm_codes, _norm_inputs, _np, _silu_limits,
                             _values)

pytestmark = gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


# 2048 items of work and more take two row groups an item: wide rows, narrow ones, odd ones.
LARGE = [(1171, 7001), (16401, 500), (40003, 130), (2051, 14336)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", LARGE)
def test_pack_of_large_matrices(shape, dtype):
    rows, cols = shape
    rng = np.random.default_rng(shape)
    t, x = _values(rng, shape, DTYPES[dtype], 10.0 ** rng.integers(-3, 3, (rows, 1)))
    t[rows // 2, cols // 2], x[rows // 2, cols // 2] = float("inf"), np.inf
    for rounding in ("rn", "sr"):
        announce("pack_i8 large", shape, dtype, rounding)
        key = dict(rounding=rounding, seed=3, step=7)
        q, s = ops.pack_i8(t, **key, base_index=11)
        padded = q if q._base is None else q._base
        assert not padded[:, cols:].any()
        if rounding == "rn":
            want_q, want_s = ol.pack(x)
            assert np.array_equal(q.cpu().numpy(), want_q)
            assert np.array_equal(to_host(s), want_s, equal_nan=True)
        step = 60 * 512 // cols + 7                     # a slice of few items
        for r in range(0, rows, rows // 9):
            part = ops.pack_i8(t[r:r + step], **key, base_index=11 + r * cols)
            assert torch.equal(part[0], q[r:r + step])
            assert torch.equal(part[1].nan_to_num(-1.0), s[r:r + step].nan_to_num(-1.0))
        for out in DTYPES.values():
            back = ops.unpack_i8(q, s, dtype=out)
            wide = s.repeat_interleave(128, 1)[:, :cols]
            want = (q.float() * wide).to(out)
            assert torch.equal(back.nan_to_num(7.0), want.nan_to_num(7.0))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("saved", ["inputs", "i8"])
@pytest.mark.parametrize("shape", [(1171, 7001), (16401, 500)])
def test_silu_mul_of_large_matrices(shape, saved, dtype):
    announce("silu_mul large", shape, saved, dtype)
    f, (rows, cols) = DTYPES[dtype], shape
    rng = np.random.default_rng(shape)
    (g, gate), (u, up) = (_values(rng, shape, f, 4.0) for _ in range(2))
    dy, dy64 = _values(rng, shape, f)

    def run(r0, r1):
        leaves = [t[r0:r1].detach().requires_grad_() for t in (g, u)]
        y = silu_mul(*leaves, saved=saved)
        return [y.detach(), *torch.autograd.grad(y, leaves, dy[r0:r1])]

    y, dgate, dup = whole = run(0, rows)
    step = 60 * 512 // cols + 7
    for r in range(0, rows, rows // 5):
        for a, b in zip(run(r, min(r + step, rows)), whole):
            assert torch.equal(a, b[r:r + step])
    _close(y, ol.silu_mul(gate, up), _silu_limits(None, gate, up, _esig(gate, f)), "y")
    if saved == "i8":
        gate, up = (ol.unpack(*ol.pack(v)).astype(np.float64) for v in (gate, up))
    dg, du = ol.silu_mul_grads(dy64, gate, up)
    _, off_g, off_u = _silu_limits(dy64, gate, up, _esig(gate, f))
    _close(dgate, dg, off_g, "dgate")
    _close(dup, du, off_u, "dup")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,dim", [(2050, 4091), (4097, 2048), (70001, 100), (1100001, 7)])
def test_lookups_of_many_tokens(n, dim, dtype):
    """Four rows a lane, the last ones past the end."""
    announce("lookup large", n, dim, dtype)
    rng = np.random.default_rng([n, dim])
    table, _ = _values(rng, (1009, dim), DTYPES[dtype])
    ids = torch.from_numpy(rng.integers(-1, 1010, n)).cuda()
    there = (ids >= 0) & (ids < 1009)
    y = embedding(ids, table, scale=3.7)
    want = (table[ids.clamp(0, 1008)].float() * np.float32(3.7)).to(DTYPES[dtype])
    assert torch.equal(y[there], want[there]) and torch.isnan(y[~there]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(15001, 40), (22007, 130), (7301, 1000), (11003, 520), (7307, 1030),
                                       (3301, 2060), (2309, 4100), (2309, 8190)])
def test_layer_norm_of_two_turns_and_more(rows, cols, dtype):
    """More rows than the chip holds at once, by two and three times: the next row's
    loads, both sets of a barrier's sums, a last turn that some of the groups have."""
    rng = np.random.default_rng([rows, cols])
    (x, dy, w, b), exact = _norm_inputs(rng, rows, cols, DTYPES[dtype], torch.float32, "wb")
    for saved in ("input", "i8"):
        announce("layer_norm turns", rows, cols, dtype, saved)
        leaves = [t.detach().requires_grad_() for t in (x, w, b)]
        y = layer_norm(*leaves, saved=saved)
        grads = torch.autograd.grad(y, leaves, dy)
        used = None
        if saved == "i8":
            want_q, want_s = ol.pack(ol.layer_norm(exact[0])[1])
            q, s = _norm_codes(x.detach(), w, b, 1e-5)
            assert np.array_equal(q.cpu().numpy()[:, :cols], want_q) and np.array_equal(s.cpu().numpy(), want_s)
            used = ol.unpack(want_q, want_s).astype(np.float64)
        # (dw, db: at most rows / 256 additions in a row, 16 groups, 68 of the join, 7 a term)
        _check_norm(*exact, 1e-5, y, *grads, used, depth=rows // 256 + 92)
        with torch.no_grad():
            assert torch.equal(layer_norm(x, w, b), y)


@pytest.mark.parametrize("n", [5000, 9000])
def test_vocabulary_of_four_passes(n):
    """Ids of 25 bits: an even number of passes, one tile and two."""
    announce("embedding of four passes", n)
    vocab = 2 ** 24 + 5
    rng = np.random.default_rng(n)
    ids = rng.integers(0, vocab, n)
    ids[::7] = vocab - 1
    ids[1::7] = rng.integers(0, 3, len(ids[1::7]))
    ids[2::7] = ids[2] + (rng.integers(0, 4, len(ids[2::7])) << 21)
    _check(ids, vocab, 1, "f32", scale=2.0, padding=1)


@pytest.mark.parametrize("n,vocab,dim", [(8192, 20000, 1000), (9001, 20000, 1000), (9001, 40000, 333)])
def test_f32_gradients_of_large_tables(n, vocab, dim):
    rng = np.random.default_rng([n, dim])
    _check(np.minimum(rng.geometric(0.0005, n) - 1, vocab - 1), vocab, dim, "f32")


def test_the_widest_rows():
    """2**24 columns: the sums' and the join's largest grids."""
    announce("embedding of 2**24 columns")
    n, vocab, dim = 33, 2, 2 ** 24
    torch.manual_seed(3)
    dy = torch.randn(n, dim, device="cuda")
    ids = torch.ones(n, dtype=torch.int64, device="cuda")
    w = torch.zeros(vocab, dim, device="cuda", requires_grad=True)
    y = embedding(ids, w)
    dw, = torch.autograd.grad(y, w, dy)
    want, size = dy.double().sum(0), dy.abs().double().sum(0)
    assert not dw[0].any() and not y.any()
    assert bool(((dw[1].double() - want).abs() <= (n + 3) * 2.0 ** -24 * size).all())


# ------------------------------------------------- what calls leave alone
class Room:
    """A marked buffer with a call's output in its middle."""
    PAD = 1024

    def __init__(self, nbytes):
        self.buf = torch.full((nbytes + 2 * self.PAD,), 0x5A, dtype=torch.uint8, device="cuda")
        self.n, self.ptr = nbytes, self.buf.data_ptr() + self.PAD

    def check(self):
        assert bool((self.buf[:self.PAD] == 0x5A).all()) and bool((self.buf[self.PAD + self.n:] == 0x5A).all())

    def as_matrix(self, dtype, rows):
        return self.buf[self.PAD:self.PAD + self.n].view(dtype).view(rows, -1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,vocab,dim", [(1025, 37, 45), (3001, 700, 131), (8191, 2000, 33), (1025, 5001, 45),
                                         (2047, 9000, 131), (8192, 40000, 7), (8193, 300, 45), (30001, 5000, 131)])
def test_embedding_gradient_writes_nothing_else(n, vocab, dim, dtype):
    """A workspace of exactly the bytes asked for: flags, zeros beside the sort, tiles."""
    announce("embedding gradient between marks", n, vocab, dim, dtype)
    f = DTYPES[dtype]
    rng = np.random.default_rng([n, vocab])
    ids = np.minimum(rng.geometric(0.01, n) - 1, vocab - 1)
    ids[n // 3:] = rng.integers(0, vocab, n - n // 3)
    t = torch.from_numpy(ids).cuda()
    dy, dy64 = _values(rng, (n, dim), f)
    need = _abi.asr_embedding_backward_workspace_bytes(n, vocab, dim)
    assert need > 0
    dw, ws = Room(vocab * dim * dy.element_size()), Room(need)
    _abi.asr_embedding_backward(t.data_ptr(), 1, n, dy.data_ptr(), dim, ops._DTYPE_CODE[f], vocab, dim, 0.5, -1,
                                dw.ptr, ws.ptr, need, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    dw.check()
    ws.check()
    _check_grad(dw.as_matrix(f, vocab), ids, dy64, vocab, 0.5, None)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(65, 203), (33, 1001), (17, 2001), (9, 4001), (5, 8001), (1300, 203),
                                       (7, 9001), (600, 8203), (130, 40007), (5, 2000003)])
@pytest.mark.parametrize("saved", ["input", "i8"])
def test_layer_norm_gradient_writes_nothing_else(rows, cols, saved, dtype):
    """One row more than one workgroup sums, more workgroups than sums, long rows."""
    announce("layer_norm gradient between marks", rows, cols, saved, dtype)
    f, st = DTYPES[dtype], torch.cuda.current_stream().cuda_stream
    rng = np.random.default_rng([rows, cols])
    (x, dy, w, b), exact = _norm_inputs(rng, rows, cols, f, torch.float32, "wb")
    size, code, ldq = x.element_size(), ops._DTYPE_CODE[f], (cols + 15) // 16 * 16
    y, stat, dx, dw, db = (Room(k) for k in (x.numel() * size, rows * 16, x.numel() * size, cols * 4, cols * 4))
    need = _abi.asr_layer_norm_backward_workspace_bytes(rows, cols)
    q, s, ws = Room(rows * ldq), Room(rows * -(-cols // 128) * 4), Room(need)
    codes = (q.ptr, ldq, s.ptr) if saved == "i8" else (None, 0, None)
    _abi.asr_layer_norm_forward(x.data_ptr(), code, cols, rows, cols, w.data_ptr(), b.data_ptr(), 0, 1e-5, y.ptr,
                                stat.ptr, *codes, st)
    _abi.asr_layer_norm_backward(dy.data_ptr(), cols, None if saved == "i8" else x.data_ptr(), cols, *codes,
                                 stat.ptr, code, rows, cols, w.data_ptr(), 0, dx.ptr, dw.ptr, db.ptr, ws.ptr, need,
                                 st)
    torch.cuda.synchronize()
    for room in (y, stat, q, s, ws, dx, dw, db):
        room.check()
    used = None
    if saved == "i8":
        used = ol.unpack(*ol.pack(ol.layer_norm(exact[0])[1])).astype(np.float64)
    _check_norm(*exact, 1e-5, y.as_matrix(f, rows), dx.as_matrix(f, rows), dw.as_matrix(torch.float32, 1)[0],
                db.as_matrix(torch.float32, 1)[0], used, depth=100)


@pytest.mark.parametrize("t,n,k", [(1, 24, 56), (67, 512, 256), (300, 77, 131), (1030, 130, 2000)])
def test_linear_keeps_no_second_copy_of_its_codes(t, n, k):
    """The forward call's workspace has w's codes and one token's room, no more."""
    announce("linear_i8 forward between marks", t, n, k)
    st = torch.cuda.current_stream().cuda_stream
    x, w = (torch.randn(*shape, device="cuda").bfloat16() for shape in ((t, k), (n, k)))
    need, ldq = _abi.asr_linear_i8_workspace_bytes(1, n, k, 0), (k + 15) // 16 * 16
    assert need <= n * (ldq + 4) + ldq + 4 + 4 * 256
    y, q, s, ws = Room(t * n * 2), Room(t * ldq), Room(t * 4), Room(need)
    _abi.asr_linear_i8_forward_saved(x.data_ptr(), k, w.data_ptr(), k, y.ptr, n, q.ptr, ldq, s.ptr, t, n, k, ws.ptr,
                                     need, st)
    torch.cuda.synchronize()
    for room in (y, q, s, ws):
        room.check()
    assert torch.equal(y.as_matrix(torch.bfloat16, t), linear_i8(x, w))
    want_q, want_s = ops.quantize_i8(x)
    assert torch.equal(q.as_matrix(torch.int8, t)[:, :k], want_q)
    assert torch.equal(s.as_matrix(torch.float32, 1)[0], want_s)
