"""The embedding and its gradient, against the definitions in binary64.

Forward: one binary32 product and its rounding, equal bits. Gradient: a row of
m tokens is m - 1 additions and two products' roundings of binary32 (u = 2**-24
each, on the magnitudes), then the rounding to its type.
"""

import numpy as np
import pytest
import torch

import oracle
from oracle import layers as ol
from adamw_optimizer_stochastic_amd import AdamWSR, _abi, embedding, layer_norm, linear_i8, silu_mul
from _gpu_util import announce, gpu, require_gpu, to_host

pytestmark = gpu
U = 2.0 ** -24
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _values(rng, shape, dtype, scale=1.0):
    t = torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(dtype)
    return t.cuda(), t.double().numpy()


def _check_grad(got, ids, dy64, vocab, scale, padding):
    want, size, count = ol.embedding_grad(ids, dy64, vocab, float(np.float32(scale)), padding)
    off = (count[:, None] + 2) * U * size
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else U
    got64 = got.double().cpu().numpy()
    bad = ~(np.abs(got64 - want) <= off + half * (np.abs(want) + off) + 2.0 ** -140)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5].tolist(), got64[bad][:5], want[bad][:5])
    assert not got64[count == 0].any()


def _run(ids, wt, dyt, scale, padding):
    leaf = wt.detach().requires_grad_()
    y = embedding(ids, leaf, scale=scale, padding_idx=padding)
    return y.detach(), torch.autograd.grad(y, leaf, dyt.view(y.shape))[0]


def _check(ids, vocab, dim, dtype, scale=1.0, padding=None, seed=0):
    announce("embedding", len(ids), vocab, dim, dtype, scale, padding)
    rng = np.random.default_rng([seed, vocab, dim])
    wt, w64 = _values(rng, (vocab, dim), DTYPES[dtype])
    dyt, dy64 = _values(rng, (len(ids), dim), DTYPES[dtype])
    outs = []
    for it in (np.int64, np.int32):
        if np.array_equal(ids.astype(it), ids):
            y, dw = _run(torch.from_numpy(ids.astype(it)).cuda(), wt, dyt, scale, padding)
            _check_grad(dw, ids, dy64, vocab, scale, padding)
            outs.append((y, dw))
    there = (ids >= 0) & (ids < vocab)
    rows = w64[ids[there]].astype(np.float32) * np.float32(scale)
    y = outs[0][0].cpu()
    assert torch.equal(y[torch.from_numpy(there)], torch.from_numpy(rows).to(DTYPES[dtype]))
    assert torch.isnan(y[torch.from_numpy(~there)]).all()
    for other in outs[1:]:
        assert torch.equal(other[1], outs[0][1])
        assert torch.equal(other[0].nan_to_num(7.0), outs[0][0].nan_to_num(7.0))
    return outs[0]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [1, 3, 8, 17, 100, 333, 2048, 2056, 4100])
def test_dims(dim, dtype):
    rng = np.random.default_rng(dim)
    for n, vocab in ((1, 1), (5, 3), (40, 1009), (200, 7)):
        _check(rng.integers(0, vocab, n), vocab, dim, dtype, scale=3.7)


@pytest.mark.parametrize("n", [1, 15, 16, 17, 1023, 1024, 1025, 2049, 4097, 8191, 8192, 8193, 16385, 30000])
@pytest.mark.parametrize("vocab", [1, 2, 200, 256, 257, 70000])
def test_tokens(n, vocab):
    """Lengths at the sort's steps; vocabularies of one to three passes."""
    rng = np.random.default_rng([n, vocab])
    _check(rng.integers(0, vocab, n), vocab, 20, "f32")


@pytest.mark.parametrize("n", [1, 255, 257, 1000, 1024, 2000, 4000, 8192, 9000])
def test_tokens_of_a_large_vocabulary(n):
    """More ids than a call of few tokens takes in one launch; zeros beside the sort."""
    rng = np.random.default_rng(n)
    ids = rng.integers(0, 140000, n)
    ids[n // 2:] = rng.integers(0, 9, n - n // 2)
    _check(ids, 140000, 20, "bf16", padding=3)


@pytest.mark.parametrize("vocab,dim", [(131072, 8), (131073, 8), (255, 300), (256, 300), (300, 2600),
                                       (70000, 30), (4096, 4096), (4097, 4096)])
def test_few_tokens(vocab, dim):
    """The single launch: ids shared out among workgroups, up to 255 each, runs of up to
    16 tokens and longer ones, at its limits of vocabulary and size."""
    rng = np.random.default_rng([vocab, dim])
    for n in (3, 700, 1024):
        ids = np.where(rng.random(n) < 0.5, rng.integers(0, vocab, n),
                       np.minimum(rng.geometric(0.03, n) - 1, vocab - 1))
        ids[:n // 10] = vocab - 1
        _check(ids, vocab, dim, "bf16" if vocab * dim > 10 ** 6 else "f32", scale=3.0)


@pytest.mark.parametrize("n", [300, 5000, 20000])
@pytest.mark.parametrize("kind", ["one", "two", "blocks", "skewed", "padded", "outside", "all outside"])
def test_repeated_and_missing_tokens(n, kind):
    """Runs of one id that end inside, at and far past a chunk's border; padding;
    ids outside the table, also very far."""
    rng = np.random.default_rng(n)
    vocab, padding = 500, None
    if kind == "one":
        ids = np.full(n, 499)
    elif kind == "two":
        ids = np.where(np.arange(n) % 3 == 0, 0, 499)
    elif kind == "blocks":
        ids = np.arange(n) // 16 % vocab
    else:
        ids = np.minimum(rng.geometric(0.02, n) - 1, vocab - 1)
    if kind == "padded":
        padding = 3
        ids[rng.random(n) < 0.6] = 3
    if kind == "outside":
        ids[::5] = -1
        ids[1::7] = vocab
        ids[2::11] = 2 ** 40 + 3
        ids[3::13] = -2 ** 33
    if kind == "all outside":
        ids = np.full(n, vocab)
    _check(ids.astype(np.int64), vocab, 260, "bf16", 16.0, padding, n)


def test_additions_in_the_tokens_order():
    """Equal calls give equal bits, and a run's sum is that of its tokens in their
    order: 1, 2**24 and -2**24 in binary32."""
    announce("embedding order")
    ids = torch.tensor([4, 2, 4, 4, 2, 2], device="cuda")
    v = torch.tensor([2.0 ** 24, 1.0, 1.0, -2.0 ** 24, 2.0 ** 24, -2.0 ** 24], device="cuda")
    w = torch.zeros(6, 9, device="cuda")
    _, dw = _run(ids, w, v[:, None].expand(6, 9).contiguous(), 1.0, None)
    assert (dw[4] == 0.0).all() and (dw[2] == 0.0).all()       # the 1 is lost in both
    v[3], v[2] = 1.0, -2.0 ** 24
    _, dw = _run(ids, w, v[:, None].expand(6, 9).contiguous(), 1.0, None)
    assert (dw[4] == 1.0).all()
    rng = np.random.default_rng(1)
    ids = torch.from_numpy(rng.integers(0, 40, 12000)).cuda()
    wt, dyt = torch.zeros(50, 300, device="cuda"), torch.randn(12000, 300, device="cuda")
    first = _run(ids, wt, dyt, 1.0, None)[1]
    for _ in range(3):
        assert torch.equal(_run(ids, wt, dyt, 1.0, None)[1], first)


def test_special_values_and_differences():
    announce("embedding special values")
    w = torch.zeros(5, 12, device="cuda")
    w[1, 3], w[2, 4] = float("inf"), float("nan")
    ids = torch.tensor([1, 2, 2, 0], device="cuda", dtype=torch.int32)
    dy = torch.ones(4, 12, device="cuda")
    dy[0, 0], dy[1, 1], dy[2, 1] = float("nan"), float("inf"), -float("inf")
    y, dw = _run(ids, w, dy, 2.0, None)
    assert torch.isinf(y[0, 3]) and torch.isnan(y[1:3, 4]).all() and torch.isfinite(y[3]).all()
    assert torch.isnan(dw[1, 0]) and torch.isnan(dw[2, 1])
    dw[1, 0] = dw[2, 1] = 0.0
    assert torch.isfinite(dw).all() and (dw[2, 2:] == 4.0).all()
    # <dy, y> is linear in w: its change along d is <dw, d>, up to the roundings of y
    rng = np.random.default_rng(2)
    ids = torch.from_numpy(rng.integers(0, 30, 90)).cuda()
    wt, w64 = _values(rng, (30, 50), torch.float32)
    dt, d64 = _values(rng, (30, 50), torch.float32)
    dyt, dy64 = _values(rng, (90, 50), torch.float32)
    moved = wt + dt
    y0, dw = _run(ids, wt, dyt, 1.5, None)
    y1, _ = _run(ids, moved, dyt, 1.5, None)
    change = np.sum(dy64 * (y1 - y0).double().cpu().numpy())
    along = (moved.double() - wt.double()).cpu().numpy()
    size = np.sum(np.abs(dy64) * (np.abs(w64[ids.cpu()]) + np.abs(d64[ids.cpu()]))) * 1.5
    assert abs(change - np.sum(dw.double().cpu().numpy() * along)) <= 100 * U * size


def test_shapes_views_empty_refusals():
    announce("embedding shapes")
    table = torch.randn(20, 40, device="cuda")
    ids = torch.arange(24, device="cuda").view(2, 3, 4) % 20
    assert torch.equal(embedding(ids, table), table[ids])
    assert torch.equal(embedding(ids.transpose(0, 2), table), table[ids.transpose(0, 2)])
    assert torch.equal(embedding(ids[0, 0, 0], table), table[0])
    leaf = table.detach().requires_grad_()
    view = leaf[:, 3:33]                                    # rows 40 apart
    y = embedding(ids[:, ::2], view, scale=2.0)
    assert torch.equal(y, 2.0 * table[ids[:, ::2]][..., 3:33])
    g, = torch.autograd.grad(y.sum(), leaf)                 # an expanded gradient
    want = torch.bincount(ids[:, ::2].reshape(-1), minlength=20).float() * 2.0
    assert torch.equal(g[:, 3:33], want[:, None].expand(20, 30)) and not g[:, :3].any()
    for shape in ((0,), (3, 0)):
        none = torch.empty(shape, dtype=torch.int64, device="cuda")
        y = embedding(none, leaf)
        assert y.shape == (*shape, 40)
        assert not torch.autograd.grad(y.sum(), leaf)[0].any()
    for vocab, dim in ((0, 5), (5, 0)):
        e = torch.empty(vocab, dim, device="cuda", requires_grad=True)
        y = embedding(torch.zeros(3, dtype=torch.int64, device="cuda"), e)
        assert y.shape == (3, dim) and torch.isnan(y).all()
        assert torch.autograd.grad(y.sum(), e)[0].shape == e.shape
    assert torch.equal(_run(ids, table, torch.ones(24, 40, device="cuda"), 1.0, -1)[1][19],
                       torch.zeros(40, device="cuda"))
    with pytest.raises(TypeError, match="int64"):
        embedding(ids.float(), table)
    with pytest.raises(ValueError, match="ids"):
        embedding(ids.cpu(), table)
    with pytest.raises(ValueError, match="padding_idx"):
        embedding(ids, table, padding_idx=20)
    with pytest.raises(ValueError, match="scale"):
        embedding(ids, table, scale=float("inf"))
    with pytest.raises(TypeError):
        embedding(ids, table.half())
    with pytest.raises(ValueError, match="V, D"):
        embedding(ids, table[0])
    held = ids.clone()
    y = embedding(held, leaf)
    held.zero_()
    with pytest.raises(RuntimeError, match="modified"):
        y.sum().backward()


def test_outputs_and_nothing_else():
    announce("embedding writes nothing else")
    n, vocab, dim, pad = 700, 37, 45, 256
    st = torch.cuda.current_stream().cuda_stream
    ids = torch.randint(0, vocab, (n,), device="cuda")
    table, dy = torch.randn(vocab, dim, device="cuda"), torch.randn(n, dim, device="cuda")
    need = _abi.asr_embedding_backward_workspace_bytes(n, vocab, dim)
    rooms = [torch.full((k + 2 * pad,), 0x5A, dtype=torch.uint8, device="cuda")
             for k in (n * dim * 4, vocab * dim * 4, need)]
    y, dw, ws = (r.data_ptr() + pad for r in rooms)
    _abi.asr_embedding_forward(ids.data_ptr(), 1, n, table.data_ptr(), 0, dim, vocab, dim, 1.0, y, st)
    _abi.asr_embedding_backward(ids.data_ptr(), 1, n, dy.data_ptr(), dim, 0, vocab, dim, 1.0, -1, dw, ws, need, st)
    torch.cuda.synchronize()
    for r in rooms:
        b = r.cpu().numpy()
        assert (b[:pad] == 0x5A).all() and (b[-pad:] == 0x5A).all()
    got = rooms[0][pad:-pad].view(torch.float32).view(n, dim)
    assert torch.equal(got, table[ids])


def test_captured_and_on_two_streams():
    announce("embedding capture")
    rng = np.random.default_rng(5)

    def data(n):
        return [torch.from_numpy(rng.integers(0, 300, n)).cuda(), _values(rng, (300, 130), torch.bfloat16)[0],
                _values(rng, (n, 130), torch.bfloat16)[0]]

    def run(ids, w, dy):
        return _run(ids, w, dy, 2.0, 7)

    for n in (900, 9000):
        cases = [data(n) for _ in range(3)]
        want = [run(*d) for d in cases]
        held = [torch.zeros_like(t) for t in cases[0]]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run(*held)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run(*held)
        for d, ref in zip(cases, want):
            for h, t in zip(held, d):
                h.copy_(t)
            graph.replay()
            torch.randn(1 << 16, device="cuda").sum().item()
            torch.cuda.synchronize()
            assert all(torch.equal(g, v) for g, v in zip(out, ref))
        streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
        torch.cuda.synchronize()
        for _ in range(4):
            for k, st in enumerate(streams):
                with torch.cuda.stream(st):
                    got[k].append(run(*cases[k]))
        torch.cuda.synchronize()
        for k in range(2):
            for o in got[k]:
                assert all(torch.equal(g, v) for g, v in zip(o, want[k]))


def test_offsets_past_32_bits():
    """A table of more than 2**31 elements: ids at both ends."""
    announce("embedding, offsets past 32 bits")
    vocab, dim = 270000, 8200
    table = torch.empty((vocab, dim), dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    for i in range(0, vocab, 30000):
        table[i:i + 30000].normal_(generator=gen)
    ids = torch.tensor([0, 269999, 262000, 1, 269999, 131072, 262144], device="cuda")
    leaf = table.requires_grad_()
    y = embedding(ids, leaf)
    assert torch.equal(y, table.detach()[ids])
    dy = torch.randn(7, dim, device="cuda").bfloat16()
    dw, = torch.autograd.grad(y, leaf, dy)
    assert torch.equal(dw[269999], (dy[1].float() + dy[4].float()).bfloat16())
    for k in (0, 2, 3, 5, 6):
        assert torch.equal(dw[ids[k]], dy[k])
    assert int((dw != 0).any(1).sum()) == 6


@pytest.mark.parametrize("saved", [False, True], ids=["inputs", "i8"])
def test_a_model_of_these_layers(saved):
    """Embedding, norm, gated MLP and the tied head in one model, its gradients
    against torch's in binary64 of the same formulas, and steps of AdamWSR.

    The int8 products are off by their codes: 1/254 of a row's largest value a
    factor, which for Gaussian rows is a relative error of about 1e-2 an operand,
    and averages over the sums. What is held is the angle and the length of each
    gradient: relative error below 0.1 (five products deep, 1e-2 sqrt(2) each at
    most, on top of bf16's 4e-3)."""
    announce("embedding to head", saved)
    rng = np.random.default_rng(6)
    vocab, dim, mlp, n = 200, 128, 256, 256
    shapes = dict(table=(vocab, dim), nw=(dim,), nb=(dim,), w1=(2 * mlp, dim), w2=(dim, mlp), fw=(dim,))
    params = {}
    for name, shape in shapes.items():
        v = rng.standard_normal(shape) * (0.1 if len(shape) == 1 else shape[-1] ** -0.5)
        v = v + 1.0 if name in ("nw", "fw") else v
        params[name] = torch.from_numpy(v.astype(np.float32)).bfloat16().cuda().requires_grad_()
    ids = torch.from_numpy(rng.integers(0, vocab, n)).cuda()
    targets = torch.roll(ids, -1)
    keep = dict(saved="i8") if saved else {}

    def model(p, step):
        h = embedding(ids, p["table"], scale=dim ** 0.5)
        z = layer_norm(h, p["nw"], p["nb"], **keep)
        z = linear_i8(z, p["w1"], seed=1, step=step, **keep)
        z = linear_i8(silu_mul(z, **keep), p["w2"], seed=2, step=step, **keep)
        z = layer_norm(h + z, p["fw"], **keep)
        return linear_i8(z, p["table"], seed=3, step=step, **keep)

    def exact(p):
        h = p["table"][ids.cpu()] * dim ** 0.5
        z = torch.nn.functional.layer_norm(h, (dim,), p["nw"], p["nb"])
        z = z @ p["w1"].t()
        z = (torch.nn.functional.silu(z[:, :mlp]) * z[:, mlp:]) @ p["w2"].t()
        z = torch.nn.functional.layer_norm(h + z, (dim,), p["fw"])
        return z @ p["table"].t()

    ref = {k: v.detach().double().cpu().requires_grad_() for k, v in params.items()}
    loss = torch.nn.functional.cross_entropy(exact(ref), targets.cpu())
    want = torch.autograd.grad(loss, list(ref.values()))
    logits = model(params, 1)
    got = torch.autograd.grad(torch.nn.functional.cross_entropy(logits.float(), targets), list(params.values()))
    for name, g, v in zip(params, got, want):
        off = float((g.double().cpu() - v).norm() / v.norm())
        assert off < 0.1, (name, off)
    opt = AdamWSR(list(params.values()), lr=1e-3, seed=0)
    for step in range(1, 4):
        opt.zero_grad()
        torch.nn.functional.cross_entropy(model(params, step).float(), targets).backward()
        opt.step()
    assert all(torch.isfinite(p).all() for p in params.values())
