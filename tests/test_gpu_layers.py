"""Layer norm, gated SiLU, 8-bit activations and the linear layer that keeps
its input in 8 bits, against the definitions in binary64.

Tolerances, with u = 2**-24 (half a step of binary32, relative): an output is
rounded once to its type (h = 2**-8 for bf16, u for f32, relative) after the
binary32 operations counted at each bound. Codes are equal.
"""

import numpy as np
import pytest
import torch

import oracle
from oracle import int8 as o8, layers as ol
from adamw_optimizer_stochastic_amd import (_abi, layer_norm, layers, linear_i8, ops, silu_mul)
from _gpu_util import announce, assert_bits_equal, gpu, require_gpu, to_host

pytestmark = gpu
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _values(rng, shape, dtype, scale=1.0):
    """A tensor of the type and its exact values in binary64."""
    t = torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(dtype)
    return t.cuda(), t.double().numpy()


def _np(t):
    return t.detach().double().cpu().numpy()


def _close(got, want, off, what):
    """|got - want| <= off, then the rounding to got's type of what is there."""
    half, got64 = HALF[got.dtype], _np(got)
    limit = off + half * (np.abs(want) + off) + 2.0 ** -140
    bad = ~(np.abs(got64 - want) <= limit)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                           got64[bad][:4], want[bad][:4], np.broadcast_to(limit, want.shape)[bad][:4])


# ----------------------------------------------------- 8-bit activations
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(1, 1), (1, 128), (3, 7), (5, 129), (2, 255), (17, 16), (33, 600),
                                   (4, 2049), (3, 2500), (700, 40)])
def test_pack(shape, dtype):
    announce("pack_i8", shape, dtype)
    rng = np.random.default_rng(shape)
    t, x = _values(rng, shape, DTYPES[dtype], 10.0 ** rng.integers(-3, 3, (shape[0], 1)))
    for rounding in ("rn", "sr"):
        q, s = ops.pack_i8(t, rounding=rounding, seed=3, step=7, base_index=11)
        want_q, want_s = ol.pack(x, rounding, 3, 7, 11)
        assert np.array_equal(q.cpu().numpy(), want_q) and q.shape == t.shape
        assert np.array_equal(to_host(s), want_s)
        padded = q._base if q._base is not None else q
        assert not padded[:, shape[1]:].any()          # the room behind a row's codes
        for out in DTYPES.values():
            back = ops.unpack_i8(q, s, dtype=out)
            want = torch.from_numpy(ol.unpack(want_q, want_s)).to(out)
            assert torch.equal(back.cpu(), want)


def test_pack_special_values():
    announce("pack_i8 special values")
    x = np.zeros((7, 300), np.float32)
    x[1, 5], x[1, 200] = np.inf, 3.0
    x[2, 299], x[2, 0] = np.nan, -1.0
    x[3] = 1e-41                                       # scales below 2**-126
    x[4, :] = -0.0
    x[5] = np.float32(3.4028235e38)
    x[6] = np.linspace(-127.5, 127.5, 300)
    t = torch.from_numpy(x).cuda()
    q, s = ops.pack_i8(t)
    want_q, want_s = ol.pack(x)
    assert np.array_equal(q.cpu().numpy(), want_q)
    assert np.array_equal(to_host(s), want_s, equal_nan=True)
    back = ops.unpack_i8(q, s, dtype=torch.float32).cpu().numpy()
    assert np.isnan(back[1, :128]).all() and np.isfinite(back[1, 128:]).all()
    assert np.isnan(back[2, 256:]).all() and np.isfinite(back[2, :256]).all()
    assert not back[3].any() and not back[4].any()


def test_pack_strided_rows_ties_and_last_positions():
    """Rows of a wider matrix from an odd column; quotients exactly half way; the
    stream's last positions."""
    announce("pack_i8 views")
    rng = np.random.default_rng(4)
    wide, x = _values(rng, (9, 1000), torch.bfloat16)
    for cols in (slice(1, 700), slice(3, 20), slice(997, 1000)):
        q, s = ops.pack_i8(wide[:, cols])
        want_q, want_s = ol.pack(x[:, cols])
        assert np.array_equal(q.cpu().numpy(), want_q) and np.array_equal(to_host(s), want_s)
    ties = np.tile(np.arange(-127, 128) / 2.0, (2, 1)).astype(np.float32)
    ties[:, [0, 128, 254]] = 127.0 / 2                 # scale 1/2: every quotient a whole number
    ties[1] = ties[1] / 2                              # and a quarter: halves
    ties[1, [0, 128, 254]] = 127.0 / 2
    q, s = ops.pack_i8(torch.from_numpy(ties).cuda())
    want_q, want_s = ol.pack(ties)
    assert np.array_equal(q.cpu().numpy(), want_q) and np.array_equal(to_host(s), want_s)
    base = 2 ** 64 - 5 * 200
    t, x = _values(rng, (5, 200), torch.float32)
    q, _ = ops.pack_i8(t, rounding="sr", seed=1, step=2, base_index=base)
    assert np.array_equal(q.cpu().numpy(), ol.pack(x, "sr", 1, 2, base)[0])
    with pytest.raises(ops.AsrError, match="2\\*\\*64"):
        ops.pack_i8(t, rounding="sr", base_index=base + 1)


def test_pack_empty_and_refusals():
    announce("pack_i8 empty")
    for shape in ((0, 5), (5, 0), (0, 0)):
        q, s = ops.pack_i8(torch.empty(shape, device="cuda"))
        assert tuple(q.shape) == shape and s.shape[0] == shape[0]
        assert tuple(ops.unpack_i8(q, s).shape) == shape
    q, s = ops.pack_i8(torch.randn(4, 100, device="cuda"))
    with pytest.raises(ValueError, match="scale"):
        ops.unpack_i8(q, s[:, :0])
    with pytest.raises((ops.AsrError, ValueError)):
        ops.unpack_i8(q.contiguous(), s)               # rows 100 bytes apart
    tight = torch.zeros(3 * 112 + 100, dtype=torch.int8, device="cuda").as_strided((4, 100), (112, 1))
    with pytest.raises(ValueError, match="room"):
        ops.unpack_i8(tight, s)
    with pytest.raises(TypeError):
        ops.unpack_i8(q.float(), s)


# ---------------------------------------------------------- layer norm
COLS = [1, 2, 7, 8, 100, 128, 129, 512, 513, 1024, 1111, 2048, 2056, 4095, 4096, 5000, 8192, 8200,
        16384, 16400, 20011]


def _norm_inputs(rng, rows, cols, dtype, wdtype, params):
    x, x64 = _values(rng, (rows, cols), dtype, 2.0)
    dy, dy64 = _values(rng, (rows, cols), dtype)
    w = w64 = b = b64 = None
    if "w" in params:
        w, w64 = _values(rng, (cols,), wdtype)
    if "b" in params:
        b, b64 = _values(rng, (cols,), wdtype)
    return (x, dy, w, b), (x64, dy64, w64, b64)


def _check_norm(x64, dy64, w64, b64, eps, y, dx, dw, db, xh_used=None, depth=80):
    """y: 8 operations of binary32. dx: sums of at most 30 additions in a row,
    7 operations a term, 5 after them (64 u covers them, on magnitudes). dw, db:
    `depth` additions in a row and 7 operations a term."""
    want, xh, rstd = ol.layer_norm(x64, w64, b64, eps)
    wide = 1.0 if w64 is None else np.abs(w64)
    _close(y, want, 8 * U * (np.abs(xh) * wide + (0 if b64 is None else np.abs(b64))), "y")
    h = xh if xh_used is None else xh_used
    gx, gw, gb = ol.layer_norm_grads(dy64, h, rstd, w64)
    g = np.abs(dy64) * wide
    if dx is not None:
        mean = lambda v: v.mean(1, keepdims=True)      # noqa: E731
        _close(dx, gx, 64 * U * rstd * (g + mean(g) + np.abs(h) * mean(g * np.abs(h))), "dx")
    if dw is not None:
        _close(dw, gw, depth * U * (np.abs(dy64) * np.abs(h)).sum(0), "dw")
    if db is not None:
        _close(db, gb, depth * U * np.abs(dy64).sum(0), "db")


def _norm_codes(x, w, b, eps):
    """The codes (with the room behind a row's) and scales that the pass keeps."""
    rows, cols = x.shape
    q, s = ops._code_buffers(rows, cols, x.device)
    y, stat = torch.empty_like(x), torch.empty(rows, 4, device="cuda")
    code = ops._DTYPE_CODE
    param = x if w is None and b is None else w if w is not None else b
    _abi.asr_layer_norm_forward(x.data_ptr(), code[x.dtype], cols, rows, cols, layers._ptr(w), layers._ptr(b),
                                code[param.dtype], eps, y.data_ptr(), stat.data_ptr(), q.data_ptr(), q.shape[1],
                                s.data_ptr(), ops._stream(x.device))
    return q, s


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("cols", COLS)
def test_layer_norm(cols, dtype, wdtype):
    for rows, params in ((1, "wb"), (3, "b"), (19, "wb"), (37, "w"), (2, "")):
        announce("layer_norm", rows, cols, dtype, wdtype, params)
        rng = np.random.default_rng([rows, cols])
        (x, dy, w, b), exact = _norm_inputs(rng, rows, cols, DTYPES[dtype], DTYPES[wdtype], params)
        leaves = [t.requires_grad_() for t in (x, w, b) if t is not None]
        for saved in ("input", "i8"):
            y = layer_norm(x, w, b, 1e-3, saved=saved)
            assert y.dtype == x.dtype and y.shape == x.shape
            grads = dict(zip([n for n, t in zip("xwb", (x, w, b)) if t is not None],
                             torch.autograd.grad(y, leaves, dy)))
            used = None
            if saved == "i8":
                xh = ol.layer_norm(exact[0], eps=1e-3)[1]
                q, s = ol.pack(xh)
                got_q, got_s = _norm_codes(x.detach(), w, b, 1e-3)
                assert np.array_equal(got_q[:, :cols].cpu().numpy(), q)
                assert np.array_equal(to_host(got_s), s)
                assert not got_q[:, cols:(cols + 15) // 16 * 16].any()
                used = ol.unpack(q, s).astype(np.float64)
            _check_norm(*exact, 1e-3, y, grads["x"], grads.get("w"), grads.get("b"), used)
            with torch.no_grad():
                assert torch.equal(layer_norm(x, w, b, 1e-3), y)


@pytest.mark.parametrize("rows,cols", [(3000, 130), (5000, 40), (2100, 1030), (1030, 2100), (530, 4200),
                                       (300, 9000)])
@pytest.mark.parametrize("saved", ["input", "i8"])
def test_layer_norm_of_many_rows(rows, cols, saved):
    """Rows for several turns of every workgroup, their number not a multiple. 256
    workgroups: at most 12 rows a lane, 16 groups, 16 shares of 16."""
    announce("layer_norm many rows", rows, cols, saved)
    rng = np.random.default_rng([rows, cols])
    (x, dy, w, b), exact = _norm_inputs(rng, rows, cols, torch.bfloat16, torch.float32, "wb")
    leaves = [t.requires_grad_() for t in (x, w, b)]
    y = layer_norm(*leaves, saved=saved)
    grads = torch.autograd.grad(y, leaves, dy)
    used = None
    if saved == "i8":
        used = ol.unpack(*ol.pack(ol.layer_norm(exact[0])[1])).astype(np.float64)
    _check_norm(*exact, 1e-5, y, *grads, used)
    again = torch.autograd.grad(layer_norm(*leaves, saved=saved), leaves, dy)
    for a, c in zip(grads, again):
        assert torch.equal(a, c)


@pytest.mark.parametrize("want", ["x", "w", "b", "xw", "wb"])
def test_layer_norm_some_gradients(want):
    announce("layer_norm gradients of", want)
    rng = np.random.default_rng(len(want))
    (x, dy, w, b), exact = _norm_inputs(rng, 40, 260, torch.float32, torch.float32, "wb")
    for name, t in zip("xwb", (x, w, b)):
        t.requires_grad_(name in want)
    y = layer_norm(x, w, b)
    got = dict(zip(want, torch.autograd.grad(y, [dict(x=x, w=w, b=b)[n] for n in want], dy)))
    _check_norm(*exact, 1e-5, y, got.get("x"), got.get("w"), got.get("b"))


def test_layer_norm_against_differences():
    """The gradients against central differences of the definition: cut off after
    h**2 f''' / 6, far below the bound, and rounded to 2**-52 |f| / h."""
    announce("layer_norm differences")
    rng = np.random.default_rng(8)
    (x, dy, w, b), (x64, dy64, w64, b64) = _norm_inputs(rng, 6, 150, torch.float32, torch.float32, "wb")
    leaves = [t.requires_grad_() for t in (x, w, b)]
    grads = [_np(g) for g in torch.autograd.grad(layer_norm(*leaves), leaves, dy)]
    for k, g in enumerate(grads):
        along = rng.standard_normal(g.shape)
        sides = []
        for h in (1e-5, -1e-5):
            moved = [x64, w64, b64]
            moved[k] = moved[k] + h * along
            sides.append(np.sum(dy64 * ol.layer_norm(*moved)[0]))
        change = (sides[0] - sides[1]) / 2e-5
        size = np.sum(np.abs(g * along))
        assert abs(change - np.sum(g * along)) <= 100 * U * size * 10 + 1e-7 * size


def test_layer_norm_special_rows():
    """Inf and NaN stay in their row (for dw and db: their sums); constant rows;
    a mean far larger than the spread; very large and small values."""
    announce("layer_norm special rows")
    rng = np.random.default_rng(9)
    x64 = rng.standard_normal((9, 200))
    x64[1, 3], x64[2, 199], x64[3, 0] = np.inf, np.nan, -np.inf
    x64[4] = 2.5
    x64[5] = x64[5] * 0.25 + 4096.0
    x64[6] *= 1e25
    x64[7] *= 1e-25
    x = torch.from_numpy(x64.astype(np.float32)).cuda().requires_grad_()
    exact = _np(x)
    for saved in ("input", "i8"):
        y = layer_norm(x, eps=1e-5, saved=saved)
        dx, = torch.autograd.grad(y, x, torch.ones_like(y).copy_(x.detach().nan_to_num(0, 0, 0).sin()))
        for r in (1, 2, 3):
            assert torch.isnan(y[r]).all() and torch.isnan(dx[r]).all()
        for r in (0, 4, 5, 6, 7, 8):
            want, xh, _ = ol.layer_norm(exact[r:r + 1])
            _close(y[r:r + 1], want, 8 * U * np.abs(xh), r)
            assert torch.isfinite(dx[r]).all()
        assert not y[4].any()
    zero = layer_norm(torch.full((2, 8), 3.0, device="cuda"), eps=0.0)
    assert torch.isnan(zero).all()                      # 0 / 0, as the formula says
    tiny = layer_norm(torch.full((2, 8), 3.0, device="cuda"), eps=0.0, saved="i8")
    assert torch.isnan(tiny).all()


def test_layer_norm_shapes_views_and_empty():
    announce("layer_norm shapes")
    rng = np.random.default_rng(10)
    base, b64 = _values(rng, (4, 5, 333), torch.bfloat16)
    w, w64 = _values(rng, (2, 150), torch.bfloat16)
    for view, exact in ((base[:, :, 1:151], b64[:, :, 1:151]), (base[:, 1:4, 7:157], b64[:, 1:4, 7:157]),
                        (base.transpose(0, 1)[:, :, :150], b64.transpose(1, 0, 2)[:, :, :150]),
                        (base[0, 0, 3:153], b64[0, 0, 3:153])):
        leaf = view.detach().requires_grad_()
        y = layer_norm(leaf, w[1])
        assert y.shape == view.shape
        want, xh, _ = ol.layer_norm(exact.reshape(-1, 150), w64[1])
        _close(y.reshape(-1, 150), want, 8 * U * np.abs(xh * w64[1]), "y")
        # an expanded gradient, and one whose rows are not contiguous
        g, = torch.autograd.grad(y.float().sum(), leaf, retain_graph=True)
        assert g.shape == leaf.shape and torch.isfinite(g).all()
    cols = base.transpose(0, 2)                         # columns 20 apart
    assert torch.equal(layer_norm(cols), layer_norm(cols.contiguous()))
    w1 = torch.randn(7, device="cuda", requires_grad=True)
    for shape in ((0, 7), (2, 0, 7), (0,), (3, 0)):
        x = torch.empty(shape, device="cuda", requires_grad=True)
        y = layer_norm(x, w1 if shape[-1] == 7 else None, saved="i8")
        assert y.shape == x.shape
        got = torch.autograd.grad(y.sum(), [x] + ([w1] if shape[-1] == 7 else []))
        assert all(not g.any() for g in got)


def test_layer_norm_refusals():
    announce("layer_norm refusals")
    x, w = torch.randn(4, 8, device="cuda"), torch.randn(8, device="cuda")
    with pytest.raises(ValueError, match="shape"):
        layer_norm(x, w[:7])
    with pytest.raises(ValueError, match="shape"):
        layer_norm(x, w[None])
    with pytest.raises(TypeError, match="same type"):
        layer_norm(x, w, w.bfloat16())
    with pytest.raises(TypeError):
        layer_norm(x.half())
    with pytest.raises(ValueError, match="on"):
        layer_norm(x, w.cpu())
    with pytest.raises(ValueError, match="dimension"):
        layer_norm(x[0, 0])
    with pytest.raises(ValueError, match="2\\*\\*24"):
        layer_norm(x[:1, :1].expand(1 << 24, 1))
    leaf = x.clone().requires_grad_()
    with torch.no_grad():
        held = leaf.clone()
    y = layer_norm(held.requires_grad_())
    with torch.no_grad():
        held.add_(1.0)
    with pytest.raises(RuntimeError, match="modified"):  # x was kept and is another now
        y.sum().backward()


# ----------------------------------------------------------- gated SiLU
def _silu_limits(dy, gate, up, esig):
    """Off by at most: sig by esig of itself (and 2**-125 where it vanishes); y two,
    du two, dg six operations of binary32 more, those of 1 + g (1 - sig) absolute."""
    sig = ol.sigmoid(gate)
    t = np.abs(1.0 + gate * (1.0 - sig))
    y = np.abs(gate * sig * up) * (esig + 4 * U) + np.abs(gate * up) * 2.0 ** -124
    if dy is None:
        return y
    du = np.abs(dy * gate * sig) * (esig + 4 * U) + np.abs(dy * gate) * 2.0 ** -124
    dg = np.abs(dy * up) * (sig * t * (esig + 6 * U) + sig * (np.abs(gate) * (sig * esig + 2 * U)
                                                              + 2 * U * (1 + np.abs(gate)))
                            + (1 + np.abs(gate)) * 2.0 ** -124)
    return y, dg, du


def _esig(gate, dtype):
    """The sigmoid's relative error: in bf16 the exponent is off by |g| 1.44 (2**-24 +
    2**-25) + 2**-23 before the instructions (2**-23 each), in f32 the functions' 4 u."""
    return (np.abs(gate) + 6) * 2.0 ** -22 if dtype == torch.bfloat16 else 8 * U


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("saved", ["inputs", "i8"])
@pytest.mark.parametrize("shape", [(1, 1), (1, 128), (3, 7), (17, 129), (5, 1000), (9, 2049), (2, 4100),
                                   (300, 24)])
def test_silu_mul(shape, saved, dtype):
    announce("silu_mul", shape, saved, dtype)
    f, (rows, cols) = DTYPES[dtype], shape
    rng = np.random.default_rng(shape)
    both, b64 = _values(rng, (rows, 2 * cols), f, 4.0)
    dy, dy64 = _values(rng, shape, f)
    gate, up = b64[:, :cols], b64[:, cols:]
    joint = both.clone().requires_grad_()
    halves = [both[:, :cols].clone().requires_grad_(), both[:, cols:].clone().requires_grad_()]
    y = silu_mul(joint, saved=saved)
    y2 = silu_mul(*halves, saved=saved)
    assert torch.equal(y, y2) and y.dtype == f and y.shape == dy.shape
    _close(y, ol.silu_mul(gate, up), _silu_limits(None, gate, up, _esig(gate, f)), "y")
    got, = torch.autograd.grad(y, joint, dy)
    got2 = torch.autograd.grad(y2, halves, dy)
    assert torch.equal(got[:, :cols], got2[0]) and torch.equal(got[:, cols:], got2[1])
    if saved == "i8":
        gate, up = (ol.unpack(*ol.pack(v)).astype(np.float64) for v in (gate, up))
    dg, du = ol.silu_mul_grads(dy64, gate, up)
    _, off_g, off_u = _silu_limits(dy64, gate, up, _esig(gate, f))
    _close(got2[0], dg, off_g, "dgate")
    _close(got2[1], du, off_u, "dup")
    with torch.no_grad():
        assert torch.equal(silu_mul(both), y)


def test_silu_mul_views_differences_and_special_values():
    announce("silu_mul views")
    rng = np.random.default_rng(21)
    base, b64 = _values(rng, (3, 4, 701), torch.float32, 3.0)
    views = [(base[:, :, 1:301], base[:, :, 350:650]), (base[:, 1:3, 3:13], base[:, 0:2, 4:14])]
    exact = [(b64[:, :, 1:301], b64[:, :, 350:650]), (b64[:, 1:3, 3:13], b64[:, 0:2, 4:14])]
    for (g, u), (g64, u64) in zip(views, exact):
        leaves = [g.detach().requires_grad_(), u.detach().requires_grad_()]
        y = silu_mul(*leaves)
        assert y.shape == g.shape
        _close(y, ol.silu_mul(g64, u64), _silu_limits(None, g64, u64, 8 * U), "y")
        dy = torch.randn(3, device="cuda")[:, None, None].expand(y.shape) if y.shape[0] == 3 else \
            torch.randn_like(y)
        got = [_np(t) for t in torch.autograd.grad(y, leaves, dy)]
        for k, v in enumerate(got):
            along = rng.standard_normal(v.shape)
            sides = []
            for h in (1e-5, -1e-5):
                moved = [g64, u64]
                moved[k] = moved[k] + h * along
                sides.append(np.sum(_np(dy) * ol.silu_mul(*moved)))
            # (the differences are cut off after h**2 f''' / 6)
            size = np.sum(np.abs(_np(dy)) * (1 + np.abs(g64)) * (1 + np.abs(u64)) * np.abs(along))
            assert abs((sides[0] - sides[1]) / 2e-5 - np.sum(v * along)) <= (100 * U + 1e-8) * size
    g = torch.tensor([[0.0, -0.0, 90.0, -90.0, -200.0, 3e38, -3e38, float("nan"), 1.0, 2.0]], device="cuda")
    u = torch.tensor([[1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, float("inf"), float("nan")]], device="cuda")
    for f in DTYPES.values():
        leaves = [g.to(f).requires_grad_(), u.to(f).requires_grad_()]
        y = silu_mul(*leaves)
        dg, du = torch.autograd.grad(y, leaves, torch.ones_like(y))
        assert torch.isfinite(y[0, :7]).all() and torch.isfinite(dg[0, :7]).all()
        assert y[0, 2] == leaves[0][0, 2] and not y[0, 4:5].any() and torch.isnan(y[0, 7])
        assert torch.isinf(y[0, 8]) and torch.isnan(y[0, 9]) and torch.isinf(dg[0, 8])
        assert torch.isfinite(du[0, :7]).all() and torch.isfinite(du[0, 8:]).all()


def test_silu_mul_empty_and_refusals():
    announce("silu_mul refusals")
    for shape in ((0, 8), (3, 0), (2, 0, 4)):
        x = torch.empty(shape, device="cuda", requires_grad=True)
        y = silu_mul(x, saved="i8")
        assert y.shape == (*shape[:-1], shape[-1] // 2)
        assert torch.autograd.grad(y.sum(), x)[0].shape == x.shape
    x = torch.randn(4, 9, device="cuda")
    with pytest.raises(ValueError, match="even"):
        silu_mul(x)
    with pytest.raises(ValueError, match="shape"):
        silu_mul(x, x[:3])
    with pytest.raises(TypeError):
        silu_mul(x, x.bfloat16())
    with pytest.raises(TypeError):
        silu_mul(x.double(), x.double())


# ----------------------------------------- the linear layer's saved codes
@pytest.mark.parametrize("shape", [(1, 16, 16), (5, 40, 24), (67, 512, 256), (130, 300, 1030), (129, 9, 300),
                                   (300, 4500, 17), (260, 260, 260)])
@pytest.mark.parametrize("grad_rounding", ["sr", "rn"])
def test_linear_saved(shape, grad_rounding):
    """Equal bits: y and dx are those of the layer that keeps x, dw the product of
    the oracle's codes of f32(dy * scale) and of x's rows."""
    t, n, k = shape
    announce("linear_i8 saved", shape, grad_rounding)
    rng = np.random.default_rng(shape)
    x, x64 = _values(rng, (t, k), torch.bfloat16)
    w, _ = _values(rng, (n, k), torch.bfloat16)
    dy, dy64 = _values(rng, (t, n), torch.bfloat16)
    x.requires_grad_(), w.requires_grad_()
    key = dict(seed=3, step=4, base_index=5, grad_rounding=grad_rounding)
    y0 = linear_i8(x, w, **key)
    dx0, = torch.autograd.grad(y0, x, dy)
    y = linear_i8(x, w, saved="i8", **key)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    assert torch.equal(y, y0) and torch.equal(dx, dx0)
    q, s = o8.quantize(x64.astype(np.float32))
    z = dy64.astype(np.float32) * s[:, None]
    qz, sz = o8.quantize(z, True, grad_rounding, 3, 4, 5)
    want = oracle.gemm_round(o8.gemm_f32(qz, q.T, sz, np.ones(k, np.float32)), "rn", 0, 0, 0)
    assert_bits_equal(to_host(dw).reshape(-1), want.reshape(-1), "dw")
    for which, alone in ((x, dx), (w, dw)):
        got, = torch.autograd.grad(linear_i8(x, w, saved="i8", **key), which, dy)
        assert torch.equal(got, alone)
    # against the formula: codes of z within a step, of x's rows within half of one
    step = 1.0 if grad_rounding == "sr" else 0.5
    z64, sx = z.astype(np.float64), s.astype(np.float64)[:, None]
    exact = dy64.T @ x64
    x_code = np.abs(x64) / sx + 0.5
    off = step * sz[:, None] * x_code.sum(0) + (np.abs(dy64).T @ (sx / 2 * np.ones((t, k)))) \
        + U * np.abs(z64).T @ x_code
    _close(dw, exact, 1.0001 * off, "dw against the formula")


def test_linear_saved_special():
    """An Inf in x, tokens of zeros, views, no tokens."""
    announce("linear_i8 saved special")
    rng = np.random.default_rng(30)
    base, b64 = _values(rng, (40, 333), torch.bfloat16)
    w, _ = _values(rng, (64, 100), torch.bfloat16)
    w.requires_grad_()
    x = base[:, 7:107].detach().requires_grad_()
    y = linear_i8(x, w, saved="i8", seed=1)
    assert torch.equal(y, linear_i8(x.detach().contiguous(), w, seed=1))
    dx, dw = torch.autograd.grad(y.float().sum(), (x, w))
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()
    with torch.no_grad():
        x[3] = 0.0
    dx, dw = torch.autograd.grad(linear_i8(x, w, saved="i8").float().sum(), (x, w))
    assert torch.isfinite(dw).all()
    with torch.no_grad():
        x[3, 5] = float("inf")
    dx, dw = torch.autograd.grad(linear_i8(x, w, saved="i8").float().sum(), (x, w))
    assert torch.isnan(dw).all() and torch.isfinite(dx).all()
    for shape in ((0, 100), (2, 0, 100)):
        e = torch.empty(shape, device="cuda", dtype=torch.bfloat16, requires_grad=True)
        y = linear_i8(e, w, saved="i8")
        dx, dw = torch.autograd.grad(y.sum(), (e, w))
        assert dx.shape == e.shape and not dw.any()
    e = torch.empty(0, 100, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    y = linear_i8(x, e, saved="i8")
    assert y.shape == (40, 0)
    dx, dw = torch.autograd.grad(y.sum(), (x, e))
    assert not dx.any() and dw.shape == e.shape


# ------------------------------------------------- what calls leave alone
def test_outputs_and_nothing_else():
    """Through the C entry points into the middle of marked buffers: every byte
    around the outputs keeps its mark."""
    announce("layers write nothing else")
    rows, cols, pad = 5, 203, 512
    st = torch.cuda.current_stream().cuda_stream
    x = torch.randn(rows, 2 * cols, device="cuda").bfloat16()
    w = torch.randn(cols, device="cuda")

    class Room:
        def __init__(self, nbytes):
            self.buf = torch.full((nbytes + 2 * pad,), 0x5A, dtype=torch.uint8, device="cuda")
            self.n = nbytes

        @property
        def ptr(self):
            return self.buf.data_ptr() + pad

        def check(self, what, written):
            torch.cuda.synchronize()
            b = self.buf.cpu().numpy()
            assert (b[:pad] == 0x5A).all() and (b[pad + self.n:] == 0x5A).all(), what
            inner = b[pad:pad + self.n].reshape(rows if written else 1, -1)
            if written and written < inner.shape[1]:
                assert (inner[:, written:] == 0x5A).all(), what

    y, q, s, stat = Room(rows * cols * 2), Room(rows * 240), Room(rows * 2 * 4), Room(rows * 16)
    _abi.asr_layer_norm_forward(x.data_ptr(), 1, 2 * cols, rows, cols, w.data_ptr(), None, 0, 1e-5, y.ptr,
                                stat.ptr, q.ptr, 240, s.ptr, st)
    for room, n in ((y, 0), (q, 208), (s, 0), (stat, 0)):
        room.check("norm forward", n)
    dx, dw, db = Room(rows * cols * 2), Room(cols * 4), Room(cols * 4)
    need = _abi.asr_layer_norm_backward_workspace_bytes(rows, cols)
    ws = Room(need)
    _abi.asr_layer_norm_backward(x.data_ptr(), 2 * cols, None, 0, q.ptr, 240, s.ptr, stat.ptr, 1, rows, cols,
                                 w.data_ptr(), 0, dx.ptr, dw.ptr, db.ptr, ws.ptr, need, st)
    for room in (dx, dw, db, ws, q, s, stat):
        room.check("norm backward", 0)
    q1, s1, q2, s2 = Room(rows * 256), Room(rows * 8), Room(rows * 256), Room(rows * 8)
    out = Room(rows * 300 * 2)
    _abi.asr_silu_mul_forward(x.data_ptr(), 2 * cols, x.data_ptr() + 2 * cols, 2 * cols, 1, rows, cols, out.ptr,
                              300, q1.ptr, s1.ptr, q2.ptr, s2.ptr, 256, st)
    for room, n in ((out, cols * 2), (q1, 208), (q2, 208), (s1, 0), (s2, 0)):
        room.check("silu forward", n)
    dg = Room(rows * 500 * 2)
    _abi.asr_silu_mul_backward(x.data_ptr(), 2 * cols, None, 0, None, 0, q1.ptr, s1.ptr, q2.ptr, s2.ptr, 256, 1,
                               rows, cols, dg.ptr, 500, dg.ptr + 2 * cols, 500, st)
    dg.check("silu backward", cols * 4)
    back = Room(rows * 300 * 4)
    _abi.asr_unpack_i8(q1.ptr, 256, s1.ptr, rows, cols, back.ptr, 0, 300, st)
    back.check("unpack", cols * 4)
    q3, s3 = Room(rows * 224), Room(rows * 8)
    _abi.asr_pack_i8(x.data_ptr(), 1, 2 * cols, rows, cols, q3.ptr, 224, s3.ptr, 0, 1, 2, 3, st)
    q3.check("pack", 208)
    s3.check("pack", 0)


# ------------------------------------------------- streams, graphs, sizes
def _step(data, saved):
    """What a block does with these operators, forward and backward."""
    x, w, b, w1, w2, dy = data
    x, w, b, w1, w2 = leaves = [t.detach().requires_grad_() for t in (x, w, b, w1, w2)]
    h = layer_norm(x, w, b, saved="i8" if saved else "input")
    h = linear_i8(h, w1, seed=1, step=2, saved="i8" if saved else "input")
    h = silu_mul(h, saved="i8" if saved else "inputs")
    y = linear_i8(h, w2, seed=2, step=2, saved="i8" if saved else "input")
    return [y.detach(), *torch.autograd.grad(y, leaves, dy)]


def _step_data(rng, rows=70):
    c, f = 130, 190
    shapes = [(rows, c), (c,), (c,), (2 * f, c), (c, f), (rows, c)]
    return [_values(rng, s, torch.bfloat16)[0] for s in shapes]


@pytest.mark.parametrize("saved", [False, True], ids=["inputs", "i8"])
def test_captured_forward_and_backward(saved):
    announce("layers capture", saved)
    rng = np.random.default_rng(40)
    data = [_step_data(rng) for _ in range(3)]
    want = [_step(d, saved) for d in data]
    held = [torch.zeros_like(t) for t in data[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(held, saved)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _step(held, saved)
    for d, ref in zip(data, want):
        for h, t in zip(held, d):
            h.copy_(t)
        graph.replay()
        torch.randn(1 << 16, device="cuda").sum().item()
        torch.cuda.synchronize()
        for g, v in zip(out, ref):
            assert torch.equal(g, v)


def test_two_streams_at_once():
    announce("layers two streams")
    rng = np.random.default_rng(41)
    data = [_step_data(rng, 400 + k) for k in range(2)]
    want = [_step(d, True) for d in data]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k].append(_step(data[k], True))
    torch.cuda.synchronize()
    for k in range(2):
        for out in got[k]:
            assert all(torch.equal(g, v) for g, v in zip(out, want[k])), k


def test_offsets_past_32_bits():
    """Matrices of more than 2**32 bytes and 2**31 elements: rows at both ends."""
    announce("layers, offsets past 32 bits")
    rows, cols = 70000, 32768
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6)
    for i in range(0, rows, 10000):
        x[i:i + 10000].normal_(generator=gen)
    pick = [0, 1, 65535, 65536, 69999]
    ends = x[pick].clone()
    q, s = ops.pack_i8(x, rounding="sr", seed=3, step=4, base_index=1)
    for r in pick:
        want = ol.pack(_np(x[r:r + 1]), "sr", 3, 4, 1 + r * cols)
        assert np.array_equal(q[r:r + 1].cpu().numpy(), want[0]) and np.array_equal(to_host(s[r:r + 1]), want[1])
    assert torch.equal(ops.unpack_i8(q, s)[pick], ops.unpack_i8(q[pick], s[pick]))
    del q, s
    small = ends.clone().requires_grad_()
    for saved in ("input", "i8"):
        leaf = x.detach().requires_grad_()
        y = layer_norm(leaf, saved=saved)
        ref = layer_norm(small, saved=saved)
        assert torch.equal(y[pick], ref)
        dx, = torch.autograd.grad(y, leaf, x)
        del y
        assert torch.equal(dx[pick], torch.autograd.grad(ref, small, ends)[0])
        del dx
    for saved in ("inputs", "i8"):
        leaf = x.detach().requires_grad_()
        y = silu_mul(leaf, saved=saved)
        ref = silu_mul(small, saved=saved)
        assert torch.equal(y[pick], ref)
        dx, = torch.autograd.grad(y, leaf, x[:, :cols // 2])
        del y
        assert torch.equal(dx[pick], torch.autograd.grad(ref, small, ends[:, :cols // 2])[0])
        del dx
