"""The int8 quantiser, product and linear layer on the GPU.

Everything here is exact, so everything is compared bit for bit: the codes and
scales with the oracle's (formed in 64 bits), the product's f32 value with
the oracle's int64 sums and binary32 products, its bf16 output with the
oracle's rounding of that value. The linear layer's outputs equal the same
products of the oracle's codes."""

import numpy as np
import pytest
import torch

import oracle
from oracle import int8 as o8
from adamw_optimizer_stochastic_amd import linear_i8, ops, workloads as wl
from _gpu_util import (gpu, require_gpu, announce, to_host, assert_bits_equal, f32_tensor,
                       bf16_tensor)

pytestmark = gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _matrix(rows, cols, dtype, seed, special=True):
    """Normal values, rows of very different size, values on code borders,
    zeros; as f32 values and as the device tensor."""
    rng = np.random.default_rng([seed, rows, cols])
    x = rng.standard_normal((rows, cols)) * 10.0 ** rng.integers(-3, 3, (rows, 1))
    if special and rows * cols > 4:
        x[rng.integers(0, rows)] = 0.0
        i = rng.integers(0, rows)
        x[i] = (rng.integers(-254, 255, cols) * 0.5)      # ties, with amax = 127
        x[i, 0] = 127.0
    x = x.astype(np.float32)
    if dtype == "bf16":
        bits = wl.f32_to_bf16_bits(x)
        return oracle.bf16_to_f32(bits).reshape(rows, cols), bf16_tensor(bits.reshape(rows, cols))
    return x, f32_tensor(x)


def _check_codes(x, t, **kw):
    q, s = ops.quantize_i8(t, **kw)
    torch.cuda.synchronize()
    want_q, want_s = o8.quantize(x, kw.get("transpose", False), kw.get("rounding", "rn"),
                                 kw.get("seed", 0), kw.get("step", 0), kw.get("base_index", 0))
    assert tuple(q.shape) == want_q.shape and q.dtype == torch.int8
    got_s = to_host(s)
    nan = np.isnan(want_s)
    assert np.array_equal(np.isnan(got_s), nan)
    assert_bits_equal(got_s[~nan], want_s[~nan], "scales")
    assert np.array_equal(q.cpu().numpy(), want_q)
    return q, s


SHAPES = [(1, 1), (1, 8), (3, 7), (5, 16), (2, 2047), (9, 2049), (4, 4096), (3, 8200), (130, 70),
          (129, 65), (257, 513), (1000, 33), (1, 9001)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("transpose", [False, True], ids=["rows", "columns"])
@pytest.mark.parametrize("shape", SHAPES)
def test_codes(shape, transpose, dtype):
    announce("quantize", shape, transpose, dtype)
    x, t = _matrix(*shape, dtype, 1)
    q, _ = _check_codes(x, t, transpose=transpose)
    if q.shape[1] % 16 and q.shape[0]:     # the padding behind every group's codes is zero
        pad = torch.as_strided(q, (q.shape[0], 16 - q.shape[1] % 16), q.stride(),
                               q.storage_offset() + q.shape[1])
        assert not bool(pad.any())
    for base in (0, 5, 2 ** 40 + 2):
        _check_codes(x, t, transpose=transpose, rounding="sr", seed=11, step=7, base_index=base)


def test_codes_of_special_values():
    announce("quantize special")
    x = np.zeros((8, 24), np.float32)
    x[1, 3], x[2, 0], x[3, 23] = np.inf, np.nan, -np.inf
    x[4] = 1e-39
    x[5, :2] = 127 * 2.0 ** -126, 2.0 ** -149
    x[6] = np.float32(3.4028234e38)
    x[7] = -0.0
    x[5, 2:] = np.linspace(0, 127 * 2.0 ** -126, 22).astype(np.float32)
    for rounding in ("rn", "sr"):
        _check_codes(x, f32_tensor(x), rounding=rounding, seed=3, step=1)
        _check_codes(np.ascontiguousarray(x.T), f32_tensor(x.T), transpose=True,
                     rounding=rounding, seed=3, step=1)


@pytest.mark.parametrize("transpose", [False, True], ids=["rows", "columns"])
def test_codes_of_strided_rows(transpose):
    """Rows with a stride, starting off 16-byte boundaries."""
    announce("quantize strided", transpose)
    x, t = _matrix(37, 83, "bf16", 2)
    for off, ld in ((0, 96), (1, 96), (3, 85)):
        store = torch.full((37 * ld + 8,), 1e9, dtype=torch.bfloat16, device="cuda")
        view = torch.as_strided(store, (37, 83), (ld, 1), off)
        view.copy_(t)
        _check_codes(x, view, transpose=transpose, rounding="sr", seed=1, step=1, base_index=1)


def test_empty_groups():
    announce("quantize empty")
    for shape, transpose in (((0, 5), False), ((5, 0), False), ((0, 5), True), ((5, 0), True)):
        x = torch.empty(shape, device="cuda")
        q, s = ops.quantize_i8(x, transpose=transpose)
        torch.cuda.synchronize()
        assert tuple(q.shape) == (shape[::-1] if transpose else shape)
        assert s.numel() == q.shape[0] and not bool(s.any())


def test_stochastic_codes_are_unbiased():
    """The mean over many keys of a code is x/s: each code is floor or ceil,
    so its standard deviation is at most 1/2, and the mean over 400 keys of
    4096 elements' errors at most 0.5 / sqrt(400 * 4096) = 3.9e-4; six of
    those, plus the 2**-17 that 16 bits leave."""
    announce("quantize unbiased")
    x, t = _matrix(4, 1024, "f32", 3, special=False)
    s = None
    total = torch.zeros(4, 1024, dtype=torch.float64, device="cuda")
    for k in range(400):
        q, s = ops.quantize_i8(t, rounding="sr", seed=k, step=2)
        total += q
    err = to_host(total) / 400 - x.astype(np.float64) / to_host(s).astype(np.float64)[:, None]
    err *= np.sign(x)
    assert abs(err.mean()) < 6 * 0.5 / np.sqrt(400 * 4096) + 2.0 ** -17


def _codes(rng, rows, k, ld, fill=77):
    """int8 operand with row stride ld, garbage behind every row's K codes."""
    full = np.full((rows, ld), fill, np.int8)
    q = rng.integers(-128, 128, (rows, k)).astype(np.int8)
    full[:, :k] = q
    return q, torch.from_numpy(full).cuda()[:, :k]


GEMM_SHAPES = [(1, 1, 1), (1, 16, 16), (1, 300, 100), (1, 4096, 4096), (2, 33, 64), (7, 130, 1000),
               (16, 257, 513), (17, 64, 128), (33, 70, 65), (64, 64, 64), (65, 63, 127),
               (100, 1000, 2049), (130, 4097, 144), (257, 259, 640), (520, 1100, 335),
               (2100, 2100, 270), (4100, 4099, 143), (4200, 4300, 160), (1500, 1500, 256)]


@pytest.mark.parametrize("shape", GEMM_SHAPES)
def test_product(shape):
    m, n, k = shape
    announce("gemm_i8", shape)
    rng = np.random.default_rng(shape)
    ld = (k + 15) // 16 * 16
    a, at = _codes(rng, m, k, ld)
    b, bt = _codes(rng, n, k, ld + 16)
    sa = (rng.random(m) * 0.1 + 1e-3).astype(np.float32)
    sb = (rng.random(n) * 1e-3).astype(np.float32)
    sat, sbt = f32_tensor(sa), f32_tensor(sb)
    want = o8.gemm_f32(a, b, sa, sb)
    for rounding, base in (("rn", 0), ("sr", 0), ("sr", 2 ** 33 + 3)):
        c32 = torch.full((m, n), np.nan, device="cuda")
        c = ops.gemm_i8(at, bt, sat, sbt, rounding=rounding, seed=9, step=4, base_index=base,
                        out_f32=c32)
        torch.cuda.synchronize()
        assert_bits_equal(to_host(c32).reshape(-1), want.reshape(-1), "f32 value")
        assert_bits_equal(to_host(c).reshape(-1),
                          oracle.gemm_round(want, rounding, 9, 4, base).reshape(-1), rounding)
        alone = ops.gemm_i8(at, bt, sat, sbt, rounding=rounding, seed=9, step=4, base_index=base)
        assert torch.equal(alone.view(torch.int16), c.view(torch.int16))


@pytest.mark.parametrize("m", [1, 5, 40, 300, 4100])
def test_product_writes_nothing_else(m):
    """Strided outputs, ragged and unaligned: what lies between the rows stays."""
    announce("gemm_i8 strided out", m)
    rng = np.random.default_rng(m)
    n, k = 4109, 48
    a, at = _codes(rng, m, k, 48)
    b, bt = _codes(rng, n, k, 64)
    sa, sb = np.ones(m, np.float32), np.full(n, 0.25, np.float32)
    want = oracle.gemm_round(o8.gemm_f32(a, b, sa, sb), "sr", 1, 2, 0)
    for ld, off in ((4112, 0), (4116, 4), (4111, 1)):
        store = torch.full((m * ld + 8,), -7.0, dtype=torch.bfloat16, device="cuda")
        out = torch.as_strided(store, (m, n), (ld, 1), off)
        ops.gemm_i8(at, bt, f32_tensor(sa), f32_tensor(sb), rounding="sr", seed=1, step=2, out=out)
        torch.cuda.synchronize()
        assert_bits_equal(to_host(out).reshape(-1), want.reshape(-1), (ld, off))
        out.fill_(-7.0)
        assert bool((store == -7.0).all())


def test_product_extremes():
    """The largest sums (K = 2**17 - 1 of -128 * -128 stays below 2**31), NaN
    scales, empty sums."""
    announce("gemm_i8 extremes")
    k = 2 ** 17 - 1
    a = torch.full((3, 2 ** 17), -128, dtype=torch.int8, device="cuda")[:, :k]
    one = torch.ones(3, device="cuda")
    c32 = torch.empty((3, 3), device="cuda")
    ops.gemm_i8(a, a, one, one, out=torch.empty((3, 3), dtype=torch.bfloat16, device="cuda"),
                out_f32=c32)
    assert bool((c32 == float(np.float32(k * 16384))).all())
    nan = torch.tensor([1.0, float("nan"), 2.0], device="cuda")
    c = ops.gemm_i8(a, a, nan, one)
    assert torch.isnan(c[1]).all() and not torch.isnan(c[[0, 2]]).any()
    empty = torch.empty((5, 0), dtype=torch.int8, device="cuda")
    five = torch.ones(5, device="cuda")
    assert not bool(ops.gemm_i8(empty, empty, five, five).any())
    assert ops.gemm_i8(empty[:0], empty, five[:0], five).shape == (0, 5)


def _bf16_of(x):
    bits = wl.f32_to_bf16_bits(np.asarray(x, np.float32))
    return oracle.bf16_to_f32(bits).reshape(x.shape), bf16_tensor(bits.reshape(x.shape))


@pytest.mark.parametrize("shape", [(1, 16, 16), (5, 40, 24), (67, 512, 256), (130, 300, 1030),
                                   (1, 4096, 1024), (300, 64, 7)])
@pytest.mark.parametrize("grad_rounding", ["sr", "rn"])
def test_linear(shape, grad_rounding):
    t, n, k = shape
    announce("linear_i8", shape, grad_rounding)
    rng = np.random.default_rng(shape)
    x, xt = _bf16_of(rng.standard_normal((t, k)))
    w, wt = _bf16_of(rng.standard_normal((n, k)) * 0.02)
    dy, dyt = _bf16_of(rng.standard_normal((t, n)) * 1e-3)
    xt.requires_grad_()
    wt.requires_grad_()
    key = dict(seed=5, step=6, base_index=7)
    y = linear_i8(xt, wt, grad_rounding=grad_rounding, **key)
    dx, dw = torch.autograd.grad(y, (xt, wt), dyt)
    torch.cuda.synchronize()

    def product(left, right):
        return oracle.gemm_round(o8.gemm_f32(left[0], right[0], left[1], right[1]), "rn")

    assert_bits_equal(to_host(y).reshape(-1),
                      product(o8.quantize(x), o8.quantize(w)).reshape(-1), "y")
    want = product(o8.quantize(dy, False, grad_rounding, 5, 6, 7), o8.quantize(w, True))
    assert_bits_equal(to_host(dx).reshape(-1), want.reshape(-1), "dx")
    want = product(o8.quantize(dy, True, grad_rounding, 5, 6, 7), o8.quantize(x, True))
    assert_bits_equal(to_host(dw).reshape(-1), want.reshape(-1), "dw")


def test_linear_gradient_of_a_sum_and_shapes():
    """A 3-D input, an expanded (broadcast) gradient, one input without a
    gradient. Each product's codes are within half a step (one step for SR)
    of the values, so y is within sum_k |x| sw/2 + |w| sx/2 + sx sw/4 of the
    exact sum, plus the bf16 rounding and three binary32 ones."""
    announce("linear_i8 shapes")
    rng = np.random.default_rng(9)
    x, xt = _bf16_of(rng.standard_normal((2, 3, 40)))
    w, wt = _bf16_of(rng.standard_normal((24, 40)))
    wt.requires_grad_()
    y = linear_i8(xt, wt, seed=1)
    assert y.shape == (2, 3, 24)
    y.float().sum().backward()
    assert wt.grad.shape == (24, 40) and xt.grad is None
    x2 = x.reshape(6, 40).astype(np.float64)
    sx = np.abs(x2).max(1)[:, None] / 127
    sw = np.abs(w.astype(np.float64)).max(1)[None, :] / 127
    bound = (np.abs(x2).sum(1)[:, None] * sw / 2 + np.abs(w).sum(1)[None, :] * sx / 2
             + 40 * sx * sw / 4)
    exact = x2 @ w.astype(np.float64).T
    got = y.detach().float().cpu().numpy().reshape(6, 24)
    assert np.all(np.abs(got - exact) <= 1.0001 * (bound + 2.0 ** -8 * (np.abs(exact) + bound)))
    # dw = dy^T x with dy all ones: the codes of dy are exact (127 each)
    dw = x2.sum(0)[None, :].repeat(24, 0)
    sc = np.abs(x2).max(0)[None, :] / 127
    err = 6 * sc / 2
    assert np.all(np.abs(wt.grad.float().cpu().numpy() - dw)
                  <= 1.0001 * (err + 2.0 ** -8 * (np.abs(dw) + err)))


@pytest.mark.parametrize("want", ["x", "w"])
@pytest.mark.parametrize("shape", [(33, 70, 50), (129, 4500, 40), (260, 130, 4200)])
def test_linear_one_gradient(shape, want):
    """Only dx or only dw, more strips of columns than a tile joins itself,
    rows with a stride; the same bits as with both."""
    t, n, k = shape
    announce("linear_i8 one gradient", shape, want)
    rng = np.random.default_rng(shape)
    x, xt = _bf16_of(rng.standard_normal((t, k)))
    w, wt = _bf16_of(rng.standard_normal((n, k)))
    dy, dyt = _bf16_of(rng.standard_normal((t, n)))
    wide = torch.zeros((t, n + 3), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:n + 2] = dyt

    def grads(need_x, need_w, d):
        a, b = xt.detach().requires_grad_(need_x), wt.detach().requires_grad_(need_w)
        y = linear_i8(a, b, seed=5, step=6, base_index=7)
        return torch.autograd.grad(y, [v for v, r in ((a, need_x), (b, need_w)) if r], d)

    dx, dw = grads(True, True, dyt)
    got = grads(want == "x", want == "w", wide[:, 2:n + 2])[0]
    torch.cuda.synchronize()
    both = dx if want == "x" else dw
    assert torch.equal(got.view(torch.int16), both.view(torch.int16))
    qd = o8.quantize(dy, want == "w", "sr", 5, 6, 7)
    q2 = o8.quantize(w if want == "x" else x, True)
    ref = oracle.gemm_round(o8.gemm_f32(qd[0], q2[0], qd[1], q2[1]), "rn")
    assert_bits_equal(to_host(got).reshape(-1), ref.reshape(-1), want)


def test_linear_empty_sums():
    announce("linear_i8 empty")
    for t, n, k in ((0, 4, 8), (4, 0, 8), (4, 8, 0), (0, 0, 0)):
        x = torch.ones((t, k), dtype=torch.bfloat16, device="cuda", requires_grad=True)
        w = torch.ones((n, k), dtype=torch.bfloat16, device="cuda", requires_grad=True)
        y = linear_i8(x, w)
        assert y.shape == (t, n) and not bool(y.any())
        dx, dw = torch.autograd.grad(y, (x, w), torch.ones_like(y))
        torch.cuda.synchronize()
        assert dx.shape == x.shape and dw.shape == w.shape
        assert not bool(dx.any()) and not bool(dw.any())


def test_codes_next_to_borders():
    """Every code border and its neighbours, for scales of every size: what the
    short way decides and what it leaves to the exact one meet here."""
    announce("quantize borders")
    rng = np.random.default_rng(8)
    rows = []
    for amax in (127.0, 1.0, 3.7e-3, 1e30, 1e-20, 2.0 ** -100, 2.0 ** -119, 0.9999999, 100.0):
        s = float(o8.scale_of(np.float32(amax)))
        v = (np.arange(0, 255) * 0.5 * s).astype(np.float32)
        v = np.concatenate([v, np.nextafter(v, np.float32(0)), np.nextafter(v, np.float32(1e38)),
                            (v * (1 + 1e-5)).astype(np.float32), (v * (1 - 1e-4)).astype(np.float32)])
        v = np.minimum(v, np.float32(amax)) * rng.choice([-1, 1], v.size).astype(np.float32)
        v[rng.integers(0, v.size)] = amax
        rows.append(v)
    x = np.stack(rows).astype(np.float32)
    for transpose in (False, True):
        y = np.ascontiguousarray(x.T) if transpose else x
        _check_codes(y, f32_tensor(y), transpose=transpose)
        for step in range(4):
            _check_codes(y, f32_tensor(y), transpose=transpose, rounding="sr", seed=2, step=step)
    small = np.where(rng.random((64, 512)) < 0.5, 2.0 ** -17, 1.0).astype(np.float32) * 127
    _check_codes(small, f32_tensor(small), rounding="sr", seed=1, step=1)


def test_other_stream_and_capture():
    """The quantiser and product on a side stream, then captured and replayed."""
    announce("int8 capture")
    rng = np.random.default_rng(4)
    x, xt = _bf16_of(rng.standard_normal((70, 300)))
    w, wt = _bf16_of(rng.standard_normal((90, 300)))

    def once():
        qx, sx = ops.quantize_i8(xt, rounding="sr", seed=1, step=2)
        qw, sw = ops.quantize_i8(wt)
        qt, st = ops.quantize_i8(xt, transpose=True)
        return ops.gemm_i8(qx, qw, sx, sw, rounding="sr", seed=3, step=4), qt, st

    want = [to_host(v) for v in once()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = once()
    side.synchronize()
    for g, v in zip(got, want):
        assert np.array_equal(to_host(g), v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = once()
    for r in range(3):
        for v in out:
            v.fill_(0)
        torch.zeros(1 << 20, device="cuda").sum().item()
        graph.replay()
        torch.cuda.synchronize()
        for g, v in zip(out, want):
            assert np.array_equal(to_host(g), v), r


def test_offsets_past_32_bits():
    """More than 2**32 elements: the codes of sampled rows and columns (whose
    stream positions pass 2**32 too) and sampled outputs of a product."""
    announce("int8 past 32 bits")
    rows, cols = 70000, 65536
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    for i in range(0, rows, 10000):
        x[i:i + 10000].normal_(generator=gen)
    pick = [0, 1, 65535, 65536, 69999]
    for rounding in ("rn", "sr"):
        q, s = ops.quantize_i8(x, rounding=rounding, seed=3, step=4, base_index=1)
        for r in pick:
            want, sw = o8.quantize(x[r:r + 1].float().cpu().numpy(), False, rounding, 3, 4,
                                   1 + r * cols)
            assert np.array_equal(q[r:r + 1].cpu().numpy(), want) and to_host(s)[r] == sw[0]
    q, s = ops.quantize_i8(x, transpose=True)
    for c in (0, 32767, 65535):
        want, sw = o8.quantize(x[:, c:c + 1].float().cpu().numpy(), True)
        assert np.array_equal(q[c:c + 1].cpu().numpy(), want) and to_host(s)[c] == sw[0]
    del x, s
    a, b = q[:, :64], q[:64000, 1024:1088]
    sa, sb = torch.rand(65536, device="cuda"), torch.rand(64000, device="cuda")
    c = ops.gemm_i8(a, b, sa, sb, rounding="sr", seed=1, step=2)
    ri, ci = [0, 1, 33000, 65535], [0, 7, 31999, 63999]
    want = o8.gemm_f32(a[ri].cpu().numpy(), b[ci].cpu().numpy(), to_host(sa)[ri], to_host(sb)[ci])
    rr, cc = np.meshgrid(ri, ci, indexing="ij")
    want = oracle.gemm_round_at(want.reshape(-1), rr.reshape(-1), cc.reshape(-1), 64000, 1, 2)
    assert_bits_equal(to_host(c[ri][:, ci]).reshape(-1), want, "sampled outputs")


def test_two_streams_at_once():
    """Two linear layers on two streams at once, forward and backward: each
    call's workspace is its own."""
    announce("linear_i8 two streams")
    rng = np.random.default_rng(6)
    layers = []
    for k in range(2):
        x, xt = _bf16_of(rng.standard_normal((400 + k, 520)))
        w, wt = _bf16_of(rng.standard_normal((610, 520)))
        dy, dyt = _bf16_of(rng.standard_normal((400 + k, 610)))
        layers.append((xt.requires_grad_(), wt.requires_grad_(), dyt))

    def run(k):
        x, w, dy = layers[k]
        y = linear_i8(x, w, seed=k)
        return [y.detach(), *torch.autograd.grad(y, (x, w), dy)]

    want = [[to_host(t) for t in run(k)] for k in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k].append(run(k))
    torch.cuda.synchronize()
    for k in range(2):
        for out in got[k]:
            for g, v in zip(out, want[k]):
                assert np.array_equal(to_host(g), v), k


def test_captured_forward_and_backward():
    """Forward and backward of the layer in one graph (on leaves of its own),
    replayed on new data."""
    announce("linear_i8 capture")
    rng = np.random.default_rng(7)
    data = [[_bf16_of(rng.standard_normal(s))[1] for s in ((70, 130), (90, 130), (70, 90))]
            for _ in range(3)]

    def run(x, w, dy):
        x, w = x.detach().requires_grad_(), w.detach().requires_grad_()
        y = linear_i8(x, w, seed=2, step=3)
        return [y.detach(), *torch.autograd.grad(y, (x, w), dy)]

    want = [[to_host(t) for t in run(*d)] for d in data]
    held = [torch.zeros_like(t) for t in data[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(*held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(*held)
    for d, ref in zip(data, want):
        for h, t in zip(held, d):
            h.copy_(t)
        graph.replay()
        torch.randn(1 << 16, device="cuda").sum().item()
        torch.cuda.synchronize()
        for g, v in zip(out, ref):
            assert np.array_equal(to_host(g), v)


def _product_bound(a, b, step_a):
    """What a product of int8 codes of a and b (rows, to one scale each) may be
    off their exact product: codes of a within step_a of a step (1/2 nearest, 1
    stochastic), of b within 1/2, then the bf16 rounding of a value that may be off
    already and three binary32 roundings (the 1.0001)."""
    sa, sb = np.abs(a).max(1)[:, None] / 127, np.abs(b).max(1)[None, :] / 127
    off = (step_a * sa * np.abs(b).sum(1)[None, :] + np.abs(a).sum(1)[:, None] * sb / 2
           + a.shape[1] * step_a * sa * sb / 2)
    return 1.0001 * (off + 2.0 ** -8 * (np.abs(a @ b.T) + off))


@pytest.mark.parametrize("grad_rounding,step", [("rn", 0.5), ("sr", 1.0)])
@pytest.mark.parametrize("shape", [(9, 17, 12), (20, 33, 24), (33, 7, 9), (70, 130, 90),
                                   (300, 33, 500)])
def test_gradients_against_formula_and_differences(shape, grad_rounding, step):
    """dx = dy w and dw = dy^T x within what their codes may be off, and against
    differences of <dy, y>: y is linear in x and in w but for the codes, so a
    step of any length does, here one along the gradient."""
    t, n, k = shape
    announce("linear_i8 gradients", shape, grad_rounding)
    rng = np.random.default_rng(shape)
    (x, xt), (w, wt), (dy, dyt) = (_bf16_of(rng.standard_normal(s))
                                   for s in ((t, k), (n, k), (t, n)))
    xt.requires_grad_(), wt.requires_grad_()
    y = linear_i8(xt, wt, seed=3, step=4, grad_rounding=grad_rounding)
    dx, dw = torch.autograd.grad(y, (xt, wt), dyt)
    x, w, dy = (v.astype(np.float64) for v in (x, w, dy))
    values = {}
    for name, got, a, b in (("y", y, x, w), ("dx", dx, dy, w.T), ("dw", dw, dy.T, x.T)):
        values[name] = got.detach().double().cpu().numpy()
        limit = _product_bound(a, b, 0.5 if name == "y" else step)
        assert np.all(np.abs(values[name] - a @ b.T) <= limit), name

    def moved(v, g):
        """v a step along g, as a bf16 tensor and its exact value."""
        return _bf16_of(v + 2 * g / np.sqrt(np.mean(g * g)))

    for name, a, b in (("dx", dy, w.T), ("dw", dy.T, x.T)):
        new, newt = moved(x if name == "dx" else w, values[name])
        x1, w1 = (new.astype(np.float64), w) if name == "dx" else (x, new.astype(np.float64))
        y1 = linear_i8(newt if name == "dx" else xt.detach(), wt.detach() if name == "dx" else newt)
        change = np.sum(dy * (y1.double().cpu().numpy() - values["y"]))
        along = x1 - x if name == "dx" else w1 - w
        limit = (np.sum(_product_bound(a, b, step) * np.abs(along))
                 + np.sum(np.abs(dy) * (_product_bound(x, w, 0.5) + _product_bound(x1, w1, 0.5))))
        if t * n * k < 20000:   # (a worst case added up over more says nothing)
            assert limit < 0.5 * abs(change)
        assert abs(change - np.sum(values[name] * along)) <= limit, name


@pytest.mark.parametrize("shape", [(65, 63, 8191), (40, 300, 1100), (40, 4500, 130), (3, 9000, 2070),
                                   (6, 5000, 500), (40, 70, 15), (700, 1700, 200), (2, 9000, 300),
                                   (64, 64, 256), (200, 100, 2 ** 17 - 1)])
def test_product_in_two_ranges_of_k(shape):
    """Products of few tiles, whose workgroups walk two ranges of K at once (the
    second one empty, shorter, or ending inside a row's last codes), and their
    neighbours that do not."""
    test_product(shape)


@pytest.mark.parametrize("ld", [4096, 4112, 8192])
@pytest.mark.parametrize("m,n,k", [(1, 8200, 2559), (1, 8200, 2561), (4, 9000, 4096), (3, 8192, 2600),
                                   (2, 16400, 2600), (5, 8200, 2600)])
def test_product_of_few_rows_and_row_strides(m, n, k, ld):
    """Up to 4 rows take one kernel or the other by how far B's rows are apart;
    the codes behind a row's K are never used."""
    announce("gemm_i8 row strides", m, n, k, ld)
    rng = np.random.default_rng([m, n, k, ld])
    a, at = _codes(rng, m, k, 4096)
    b, bt = _codes(rng, n, k, ld)
    sa, sb = rng.random(m).astype(np.float32), rng.random(n).astype(np.float32)
    c32 = torch.full((m, n), np.nan, device="cuda")
    c = ops.gemm_i8(at, bt, f32_tensor(sa), f32_tensor(sb), rounding="sr", seed=3, step=1, out_f32=c32)
    torch.cuda.synchronize()
    want = o8.gemm_f32(a, b, sa, sb)
    assert_bits_equal(to_host(c32).reshape(-1), want.reshape(-1), "f32 value")
    assert_bits_equal(to_host(c).reshape(-1), oracle.gemm_round(want, "sr", 3, 1, 0).reshape(-1), "sr")


def test_last_positions():
    """Positions up to the last one, 2**64 - 1 (a run of 8 that goes past a row's
    end draws from position 0 on, and uses none of it)."""
    announce("int8 last positions")
    x, t = _matrix(5, 70, "f32", 12)
    top = 2 ** 64 - 5 * 70
    for transpose in (False, True):
        _check_codes(x, t, transpose=transpose, rounding="sr", seed=4, step=9, base_index=top)
    rng = np.random.default_rng(12)
    for m, n, k in ((3, 37, 600), (70, 65, 40)):
        a, at = _codes(rng, m, k, (k + 15) // 16 * 16)
        b, bt = _codes(rng, n, k, (k + 15) // 16 * 16)
        sa, sb = rng.random(m).astype(np.float32), rng.random(n).astype(np.float32)
        base = 2 ** 64 - m * n
        c = ops.gemm_i8(at, bt, f32_tensor(sa), f32_tensor(sb), rounding="sr", seed=4, step=9,
                        base_index=base)
        want = oracle.gemm_round(o8.gemm_f32(a, b, sa, sb), "sr", 4, 9, base)
        assert_bits_equal(to_host(c).reshape(-1), want.reshape(-1), (m, n, k))
        with pytest.raises(ops.AsrError, match="2\\*\\*64"):
            ops.gemm_i8(at, bt, f32_tensor(sa), f32_tensor(sb), rounding="sr", seed=4, step=9,
                        base_index=base + 1)
