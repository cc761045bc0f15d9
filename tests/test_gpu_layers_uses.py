"""The layers and 8-bit activations at the borders of their kernels' choices and
in the ways that a program uses them: inputs given twice, gradients spread over
rows, gradients of gradients, changed saved tensors, inference.

u = 2**-24, half a step of binary32; codes and repeated calls are equal bits.
"""

import numpy as np
import pytest
import torch

from oracle import int8 as o8, layers as ol
from adamw_optimizer_stochastic_amd import _abi, embedding, layer_norm, linear_i8, ops, silu_mul
from _gpu_util import announce, gpu, require_gpu, to_host
from test_gpu_layers import DTYPES, U, _check_norm, _close, _norm_inputs, _np, _values

pytestmark = gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("rounding", ["rn", "sr"])
@pytest.mark.parametrize("exponent", [-119, -100, -60, -54, -53, -1, 0, 100, 120])
def test_codes_next_to_the_borders(exponent, rounding):
    """Blocks for every 8-bit mantissa of the largest value, the others few-bit values
    next to it: ratios that are ties but for the scale's rounding. Both sides of the
    scale below which a group is scaled (2**-60)."""
    announce("codes next to borders", exponent, rounding)
    rng = np.random.default_rng([exponent + 200, len(rounding)])
    top = (128 + np.arange(128))[:, None] * 2.0 ** (exponent - 7)
    x = top * rng.integers(-16, 17, (128, 128)) / 2.0 ** rng.integers(4, 8, (128, 128))
    x[:, 0] = top[:, 0]
    x[:, 64:] = np.clip((128 + rng.integers(0, 128, (128, 64))) * 2.0 ** (exponent - 7)
                        / 2.0 ** rng.integers(0, 8, (128, 64)), 0, top)
    for dtype in DTYPES.values():
        t = torch.from_numpy(x.astype(np.float32)).to(dtype).cuda()
        x32 = _np(t).astype(np.float32)
        q, s = ops.pack_i8(t, rounding=rounding, seed=5, step=6, base_index=7)
        want_q, want_s = ol.pack(x32, rounding, 5, 6, 7)
        assert np.array_equal(to_host(s), want_s) and np.array_equal(q.cpu().numpy(), want_q)
        key = dict(rounding=rounding, seed=5, step=6, base_index=7)
        q, s = ops.quantize_i8(t, **key)
        want_q, want_s = o8.quantize(x32, **key)
        assert np.array_equal(to_host(s), want_s) and np.array_equal(q.cpu().numpy(), want_q)


@pytest.mark.parametrize("cols,groups", [(500, 16), (1000, 8), (2000, 4), (4000, 2), (8000, 1)])
@pytest.mark.parametrize("saved", ["input", "i8"])
def test_layer_norm_gradients_by_one_workgroup_and_two(cols, groups, saved):
    """Rows of one to five turns of a workgroup, which sums up to four by itself."""
    for rows in (groups, groups + 1, 4 * groups, 4 * groups + 1, 5 * groups):
        announce("layer_norm turns", rows, cols, saved)
        rng = np.random.default_rng([rows, cols])
        (x, dy, w, b), exact = _norm_inputs(rng, rows, cols, torch.bfloat16, torch.float32, "wb")
        leaves = [t.requires_grad_() for t in (x, w, b)]
        grads = torch.autograd.grad(layer_norm(*leaves, saved=saved), leaves, dy)
        used = None
        if saved == "i8":
            used = ol.unpack(*ol.pack(ol.layer_norm(exact[0])[1])).astype(np.float64)
        _check_norm(*exact, 1e-5, layer_norm(x, w, b), *grads, used)
        only, = torch.autograd.grad(layer_norm(*leaves, saved=saved), x, dy)
        assert torch.equal(only, grads[0])


def test_inputs_given_twice():
    """Gradients of every place that a tensor has are added (by torch, in f32: u of
    the sum more)."""
    announce("inputs given twice")
    rng = np.random.default_rng(60)
    x, x64 = _values(rng, (33, 200), torch.float32)
    dy, dy64 = _values(rng, (33, 200), torch.float32)
    x.requires_grad_()
    sig = 1 / (1 + np.exp(-x64))
    up, gate = dy64 * x64 * sig, dy64 * x64 * sig * (1 + x64 * (1 - sig))
    y = silu_mul(x, x)
    # (u of a handful of f32 operations, expf's 2 u among them, on magnitudes)
    _close(y, x64 * x64 * sig, 12 * U * x64 * x64, "y")
    _close(torch.autograd.grad(y, x, dy)[0], up + gate,
           32 * U * (np.abs(up) + np.abs(dy64 * x64) * (1 + np.abs(x64))), "dx")
    w, w64 = _values(rng, (200,), torch.float32)
    w.requires_grad_()
    dw, = torch.autograd.grad(layer_norm(x, w, w), w, dy)
    _, xh, _ = ol.layer_norm(x64)
    _close(dw, (dy64 * xh).sum(0) + dy64.sum(0), 80 * U * (np.abs(dy64) * (1 + np.abs(xh))).sum(0), "dw")
    # the norm of its own weight
    v, v64 = _values(rng, (200,), torch.float32)
    v.requires_grad_()
    one = dy[:1].reshape(200)
    dv, = torch.autograd.grad(layer_norm(v, v), v, one)
    _, xh, rstd = ol.layer_norm(v64[None])
    gx, gw, _ = ol.layer_norm_grads(dy64[:1], xh, rstd, v64)
    g = np.abs(dy64[0] * v64)
    _close(dv, gx[0] + gw, 64 * U * (rstd[0] * (g + g.mean() + np.abs(xh[0]) * (g * np.abs(xh[0])).mean())
                                     + np.abs(dy64[0] * xh[0])), "dv")
    ids = torch.from_numpy(rng.integers(0, 50, 64)).cuda()
    table, _ = _values(rng, (50, 40), torch.float32)
    table.requires_grad_()
    dy2, _ = _values(rng, (64, 40), torch.float32)
    a, = torch.autograd.grad(embedding(ids, table), table, dy2)
    both, = torch.autograd.grad(embedding(ids, table) + embedding(ids, table, scale=2.0), table, dy2)
    c, = torch.autograd.grad(embedding(ids, table, scale=2.0), table, dy2)
    assert torch.equal(both, a + c)


def _calls(rng):
    """(name, function of a tensor, leaf) of each operator, both ways of saving."""
    x = _values(rng, (20, 256), torch.bfloat16)[0]
    w = _values(rng, (256,), torch.bfloat16)[0]
    m = _values(rng, (64, 256), torch.bfloat16)[0]
    ids = torch.from_numpy(rng.integers(0, 20, (5, 7))).cuda()
    out = [("embedding", lambda t: embedding(ids, t), x)]
    for saved in (False, True):
        out += [("norm %d" % saved, lambda t, k="i8" if saved else "input": layer_norm(t, w, saved=k), x),
                ("silu %d" % saved, lambda t, k="i8" if saved else "inputs": silu_mul(t, saved=k), x),
                ("linear %d" % saved, lambda t, k="i8" if saved else "input": linear_i8(t, m, saved=k), x)]
    return out


def test_gradients_spread_over_rows():
    """A sum's gradient, one number for all places, is the same as written out."""
    announce("spread gradients")
    for name, f, x in _calls(np.random.default_rng(61)):
        leaf = x.clone().requires_grad_()
        y = f(leaf)
        spread = torch.ones((), dtype=y.dtype, device="cuda").expand(y.shape)
        got, = torch.autograd.grad(y, leaf, spread)
        want, = torch.autograd.grad(f(leaf), leaf, torch.ones_like(y))
        assert torch.equal(got, want), name
        by_columns = torch.ones_like(y.transpose(0, -1)).contiguous().transpose(0, -1)
        got, = torch.autograd.grad(f(leaf), leaf, by_columns)
        assert torch.equal(got, want), name


def test_gradients_of_gradients_are_refused():
    announce("second gradients")
    for name, f, x in _calls(np.random.default_rng(62)):
        leaf = x.clone().requires_grad_()
        y = f(leaf)
        dy = torch.ones_like(y).requires_grad_()
        first, = torch.autograd.grad(y, leaf, dy, create_graph=True)
        want, = torch.autograd.grad(f(leaf), leaf, torch.ones_like(y))
        assert torch.equal(first, want), name
        with pytest.raises(RuntimeError, match="twice"):
            first.float().sum().backward()


def test_changed_inputs_are_noticed():
    """What the backward pass reads again may not have been written in between; what
    it keeps codes of may."""
    announce("changed inputs")
    rng = np.random.default_rng(63)
    for name, f, x in _calls(rng):
        leaf = x.clone().requires_grad_()
        held = leaf * 1.0
        want, = torch.autograd.grad(f(held), held, torch.ones_like(f(held)))
        y = f(held)
        held.mul_(2.0)
        if name.endswith("0"):
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                torch.autograd.grad(y, leaf, torch.ones_like(y))
        else:
            got, = torch.autograd.grad(y, leaf, torch.ones_like(y))
            assert torch.equal(got, want), name
    ids = torch.zeros(9, dtype=torch.int64, device="cuda")
    table = torch.randn(5, 8, device="cuda", requires_grad=True)
    y = embedding(ids, table)
    ids.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_inference_gives_the_same():
    announce("inference")
    for name, f, x in _calls(np.random.default_rng(64)):
        want = f(x.clone().requires_grad_())
        with torch.inference_mode():
            got = f(x.clone())
        assert not got.requires_grad and torch.equal(got, want), name
        with torch.no_grad():
            assert torch.equal(f(x.clone().requires_grad_()), want), name


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(3, 7), (700, 1000), (5, 4096), (40, 5001), (3, 9001)])
def test_outputs_in_their_inputs_place(rows, cols, dtype):
    """The overlaps that the interface allows: y in x's, gate's or up's place, the
    gradients of gate and up in those of dy, gate and up."""
    announce("in place", rows, cols, dtype)
    rng = np.random.default_rng([rows, cols])
    a, b, c = (_values(rng, (rows, cols), DTYPES[dtype])[0] for _ in range(3))
    w = _values(rng, (cols,), DTYPES[dtype])[0]
    code, st = ops._DTYPE_CODE[a.dtype], ops._stream(a.device)
    x = a.clone()
    _abi.asr_layer_norm_forward(x.data_ptr(), code, cols, rows, cols, w.data_ptr(), None, code, 1e-5,
                                x.data_ptr(), None, None, 0, None, st)
    assert torch.equal(x, layer_norm(a, w))
    want = silu_mul(a, b)
    for place in range(2):
        g, u = a.clone(), b.clone()
        _abi.asr_silu_mul_forward(g.data_ptr(), cols, u.data_ptr(), cols, code, rows, cols,
                                  (g, u)[place].data_ptr(), cols, None, None, None, None, 0, st)
        assert torch.equal((g, u)[place], want) and torch.equal((u, g)[place], (b, a)[place])
    leaves = [a.clone().requires_grad_(), b.clone().requires_grad_()]
    want = torch.autograd.grad(silu_mul(*leaves), leaves, c)
    for first, second in ((0, 1), (1, 2), (2, 0), (1, 0)):
        t = [c.clone(), a.clone(), b.clone()]          # dy, gate, up
        _abi.asr_silu_mul_backward(t[0].data_ptr(), cols, t[1].data_ptr(), cols, t[2].data_ptr(), cols,
                                   None, None, None, None, 0, code, rows, cols, t[first].data_ptr(), cols,
                                   t[second].data_ptr(), cols, st)
        assert torch.equal(t[first], want[0]) and torch.equal(t[second], want[1])


def test_many_layers_at_once_on_many_threads():
    """Calls from several threads, each on a stream of its own."""
    announce("threads")
    import threading
    calls = _calls(np.random.default_rng(65))
    want = []
    for name, f, x in calls:
        leaf = x.clone().requires_grad_()
        y = f(leaf)
        want.append((y, torch.autograd.grad(y, leaf, torch.ones_like(y))[0]))
    torch.cuda.synchronize()
    wrong = []

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(5):
                for (name, f, x), (y0, d0) in zip(calls, want):
                    leaf = x.detach().requires_grad_()
                    y = f(leaf)
                    d, = torch.autograd.grad(y, leaf, torch.ones_like(y))
                    torch.cuda.current_stream().synchronize()
                    if not (torch.equal(y, y0) and torch.equal(d, d0)):
                        wrong.append(name)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not wrong and not any(t.is_alive() for t in threads)


@pytest.mark.parametrize("saved", ["input", "i8"])
@pytest.mark.parametrize("rows,cols", [(1, 64), (37, 1111), (300, 4100), (5, 9001)])
def test_layer_norm_of_f32_with_bf16_weights(rows, cols, saved):
    announce("layer_norm f32, bf16 weights", rows, cols, saved)
    rng = np.random.default_rng([rows, cols])
    (x, dy, w, b), exact = _norm_inputs(rng, rows, cols, torch.float32, torch.bfloat16, "wb")
    leaves = [t.requires_grad_() for t in (x, w, b)]
    y = layer_norm(*leaves, saved=saved)
    grads = torch.autograd.grad(y, leaves, dy)
    assert y.dtype == torch.float32 and [g.dtype for g in grads] == [t.dtype for t in leaves]
    used = None
    if saved == "i8":
        used = ol.unpack(*ol.pack(ol.layer_norm(exact[0])[1])).astype(np.float64)
    _check_norm(*exact, 1e-5, y, *grads, used)


@pytest.mark.parametrize("saved", ["input", "i8"])
def test_linear_of_no_tokens_and_for_some_gradients(saved):
    announce("linear, no tokens, some gradients", saved)
    rng = np.random.default_rng(66)
    x, w = (_values(rng, s, torch.bfloat16)[0].requires_grad_() for s in ((40, 100), (60, 100)))
    dy = _values(rng, (40, 60), torch.bfloat16)[0]
    dx, dw = torch.autograd.grad(linear_i8(x, w, seed=1, saved=saved), (x, w), dy)
    for one, want in ((x, dx), (w, dw)):
        y = linear_i8(*(t if t is one else t.detach() for t in (x, w)), seed=1, saved=saved)
        assert torch.equal(torch.autograd.grad(y, one, dy)[0], want)
    strided = torch.zeros((40, 133), dtype=torch.bfloat16, device="cuda")[:, 7:107].copy_(x.detach()).requires_grad_()
    y = linear_i8(strided, w.detach().t().contiguous().t().requires_grad_(), seed=1, saved=saved)
    assert torch.equal(torch.autograd.grad(y, strided, dy)[0], dx)
    none = torch.empty((0, 100), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    y = linear_i8(none, w, saved=saved)
    dx, dw = torch.autograd.grad(y, (none, w), torch.empty_like(y))
    assert y.shape == (0, 60) and dx.shape == (0, 100) and dw.shape == w.shape and not dw.any()


def test_layer_norm_of_rows_far_from_zero_and_of_one_value():
    """Means of 1e6 times the spread, constant rows, one column, and values of the
    type's whole range (differences that stay in it)."""
    announce("layer_norm far from zero")
    rng = np.random.default_rng(67)
    x = rng.standard_normal((6, 1000)).astype(np.float32)
    x[0] += np.float32(1e6)
    x[1] = np.float32(-3e5)
    x[2] *= np.float32(1e37)
    x[3] *= np.float32(1e-30)
    x[4, 1:] = np.float32(1e-3)
    x[5] = np.where(rng.random(1000) < 0.5, np.float32(1.5e38), np.float32(-1.5e38))
    t = torch.from_numpy(x).cuda()
    for saved in ("input", "i8"):
        leaf = t.clone().requires_grad_()
        y = layer_norm(leaf, saved=saved)
        dy, dy64 = _values(rng, x.shape, torch.float32)
        dx, = torch.autograd.grad(y, leaf, dy)
        used = None
        if saved == "i8":
            used = ol.unpack(*ol.pack(ol.layer_norm(x.astype(np.float64))[1])).astype(np.float64)
        _check_norm(x.astype(np.float64), dy64, None, None, 1e-5, y, dx, None, None, used)


@pytest.mark.parametrize("saved", ["input", "i8"])
@pytest.mark.parametrize("rows,cols", [(1023, 8200), (1024, 8200), (1030, 9001), (3, 16385), (2, 40007), (1, 200000)])
def test_layer_norm_of_long_rows(rows, cols, saved):
    """Both numbers of lanes, rows that end in a lane's first and second run. (depth:
    four rows a share, 64 shares of 4; a row's sums are in 64 bits.)"""
    announce("layer_norm long rows", rows, cols, saved)
    rng = np.random.default_rng([rows, cols])
    (x, dy, w, b), exact = _norm_inputs(rng, rows, cols, torch.bfloat16, torch.bfloat16, "wb")
    leaves = [t.requires_grad_() for t in (x, w, b)]
    y = layer_norm(*leaves, saved=saved)
    grads = torch.autograd.grad(y, leaves, dy)
    used = None
    if saved == "i8":
        used = ol.unpack(*ol.pack(ol.layer_norm(exact[0])[1])).astype(np.float64)
    _check_norm(*exact, 1e-5, y, *grads, used)
