"""Newton-Schulz orthogonalisation, the Muon step and MuonSR on the GPU.

The oracle computes the definition in 64 bits, and apart from it what the
scheme's roundings (f16 operands, X in two f16 parts) cost on the same input.
The kernel makes the same roundings of sums that differ in their last f32 bits,
so a rounding may fall the other way: its error is held to twice the
scheme's own, plus the bf16 rounding of the result (at most 2**-8 of every
value, so of the Frobenius norm) and 2**-18 for the f32 sums (K = 2**12 terms
or fewer between cancelling terms) where the scheme's error is next to
nothing."""

import numpy as np
import pytest
import torch

import oracle
from oracle import muon as om
from adamw_optimizer_stochastic_amd import MuonSR, AdamWSR, linear_i8, ops
from _gpu_util import gpu, require_gpu, announce, to_host, assert_bits_equal

pytestmark = gpu

SUMS = 2.0 ** -18


def _scheme_error(u, want, **kw):
    """What the kernel's result may be off before its own rounding, relative to
    `want`. A matrix of one row has one singular value, whose few roundings do
    not average, so the scheme's error on it is a single draw; its bound:
    s -> s (a + B), B = b A + c A^2, A = s^2. With |B| <= 2.81 and |b A + 2 c A^2| <=
    1.55 on s in [0.7, 1.2], the roundings of A (with its operands'), of B and
    of the operand beside B move a step by at most 1.2 (3 * 1.55 + 2 * 2.81) 2**-11 =
    6e-3; from s = 1 the orbit is 0.701, 1.114, 0.721, 1.089, 0.70, with slopes
    -1.142, 1.31, -1.257, 0.745 behind its first four steps, so five steps' errors add up
    to at most 5.3 * 6e-3 = 3.2e-2, of 0.70: 1/16 covers it to second order."""
    if min(u.shape) == 1:
        return 2.0 ** -4
    return 2 * om.relative(om.newton_schulz_f16(u, **kw), want) + SUMS


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _matrix(kind, rows, cols, seed=0, dtype=torch.bfloat16):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + rows * 131 + cols)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    if kind == "normal":
        x = normal(rows, cols)
    elif kind == "lowrank":
        r = max(1, min(rows, cols) // 16)
        x = normal(rows, r) @ normal(r, cols)
    else:   # strong directions over a floor
        r = max(1, min(rows, cols) // 16)
        x = normal(rows, r) @ normal(r, cols) / r ** 0.5 + 0.1 * normal(rows, cols)
    return (x * 1e-3).to(dtype).contiguous()


SHAPES = [(1, 1), (1, 7), (7, 1), (16, 16), (64, 64), (65, 64), (64, 65), (33, 130), (130, 33),
          (128, 256), (517, 333), (200, 1030), (1030, 200), (700, 700), (1, 4099), (2049, 3)]


@pytest.mark.parametrize("kind", ["normal", "lowrank", "floor"])
@pytest.mark.parametrize("shape", SHAPES)
def test_newton_schulz(shape, kind):
    announce("newton_schulz", shape, kind)
    for dtype in (torch.bfloat16, torch.float32):
        g = _matrix(kind, *shape, dtype=dtype)
        o = ops.newton_schulz(g)
        torch.cuda.synchronize()
        want = om.newton_schulz(g)
        tol = _scheme_error(g, want) + 2.0 ** -8
        assert om.relative(o, want) <= tol


@pytest.mark.parametrize("shape", [(16, 1024, 1024), (16, 1536, 512), (12, 1600, 1700),
                                   (3, 300, 2000), (40, 48, 64), (1, 4352, 4096),
                                   (8, 1024, 2000), (2, 2048, 2048)])
def test_batches(shape):
    """Every tile (the number of tiles picks it) and more matrices than one
    launch takes; each matrix's result is that of the matrix alone, bit for
    bit."""
    announce("newton_schulz batch", shape)
    b, rows, cols = shape
    g = torch.stack([_matrix("floor", rows, cols, seed=k) for k in range(b)])
    o = ops.newton_schulz(g)
    torch.cuda.synchronize()
    for k in sorted({0, b // 2, b - 1}):
        want = om.newton_schulz(g[k])
        tol = 2 * om.relative(om.newton_schulz_f16(g[k]), want) + 2.0 ** -8 + SUMS
        assert om.relative(o[k], want) <= tol, k
        alone = ops.newton_schulz(g[k])
        assert torch.equal(alone.view(torch.int16), o[k].view(torch.int16)), k
    # in place, and on an unaligned view
    h = g.clone()
    ops.newton_schulz(h, out=h)
    assert torch.equal(h.view(torch.int16), o.view(torch.int16))
    store = torch.empty(g.numel() + 1, dtype=torch.bfloat16, device="cuda")
    view = store[1:].view(g.shape)
    view.copy_(g)
    again = torch.empty_like(store)
    ops.newton_schulz(view, out=again[1:].view(g.shape))
    assert torch.equal(again[1:].view(torch.int16), o.reshape(-1).view(torch.int16))


def test_symmetry_and_steps():
    """A transposed matrix gives the transposed result; other step counts and
    coefficients."""
    announce("newton_schulz variants")
    g = _matrix("floor", 190, 260)
    o, ot = ops.newton_schulz(g), ops.newton_schulz(g.t().contiguous())
    assert torch.equal(o.view(torch.int16), ot.t().contiguous().view(torch.int16))
    for steps, c in ((1, om.COEFFICIENTS), (2, om.COEFFICIENTS), (8, (1.875, -1.25, 0.375))):
        want = om.newton_schulz(g, steps, c)
        tol = 2 * om.relative(om.newton_schulz_f16(g, steps, c), want) + 2.0 ** -8 + SUMS
        assert om.relative(ops.newton_schulz(g, steps=steps, coefficients=c), want) <= tol


def test_special_matrices():
    announce("newton_schulz special")
    assert not bool(ops.newton_schulz(torch.zeros(40, 70, device="cuda")).any())
    for bad in (float("inf"), float("nan")):
        g = torch.randn(70, 40, device="cuda")
        g[3, 5] = bad
        both = torch.stack([torch.ones(70, 40, device="cuda"), g])
        o = ops.newton_schulz(both)
        assert torch.isnan(o[1]).all() and torch.isfinite(o[0]).all()
    # the norm of huge and of tiny values, in one element and in many
    for scale in (1e38, 1e-30):
        g = torch.randn(30, 50, device="cuda").clamp(-3, 3) * scale
        want = om.newton_schulz(g, eps=0.0)
        o = ops.newton_schulz(g, eps=0.0)
        tol = 2 * om.relative(om.newton_schulz_f16(g, eps=0.0), want) + 2.0 ** -8 + SUMS
        assert om.relative(o, want) <= tol
    one = torch.zeros(300, 500, device="cuda")
    one[17, 333] = -5.0
    o = ops.newton_schulz(one)
    want = om.newton_schulz(one)
    assert om.relative(o, want) <= 2.0 ** -8 + 2 * om.relative(om.newton_schulz_f16(one), want) + SUMS
    assert ops.newton_schulz(torch.empty(0, 5, device="cuda")).shape == (0, 5)
    assert ops.newton_schulz(torch.empty(0, 4, 5, device="cuda")).shape == (0, 4, 5)
    # eps that matters: a norm next to it
    g = torch.full((8, 8), 1e-8, device="cuda")
    want = om.newton_schulz(g)
    assert om.relative(ops.newton_schulz(g), want) <= (
        2 * om.relative(om.newton_schulz_f16(g), want) + 2.0 ** -8 + SUMS)


MUON_SHAPES = [(1, 1), (64, 64), (100, 37), (37, 100), (256, 264), (130, 515)]


def _state(shapes, pt, gt, seed=0):
    ps = [(_matrix("normal", *s, seed=seed + i, dtype=torch.float32) * 20).to(pt)
          for i, s in enumerate(shapes)]
    gs = [_matrix("floor", *s, seed=seed + 50 + i, dtype=torch.float32).to(gt)
          for i, s in enumerate(shapes)]
    ms = [_matrix("floor", *s, seed=seed + 90 + i, dtype=torch.float32) for i, s in enumerate(shapes)]
    return ps, gs, ms


@pytest.mark.parametrize("nesterov", [True, False], ids=["nesterov", "plain"])
@pytest.mark.parametrize("gt", [torch.bfloat16, torch.float32], ids=["gbf16", "gf32"])
def test_muon_step(gt, nesterov):
    """f32 parameters within the orthogonalisation's error of the 64-bit step
    (plus three f32 roundings); the momentum exact; bf16 parameters exactly the
    RN and SR roundings of what f32 parameters of the same values become."""
    announce("muon_step", gt, nesterov)
    shapes = MUON_SHAPES + [(64, 64)]
    ps, gs, ms = _state(shapes, torch.bfloat16, gt)
    bases = [5 + 1000 * i for i in range(len(shapes))]
    hp = dict(lr=0.02, momentum=0.9, nesterov=nesterov, weight_decay=0.1, step=3, seed=11)
    p32 = [p.float() for p in ps]
    m32 = [m.clone() for m in ms]
    ops.muon_step(p32, gs, m32, bases, **hp)
    torch.cuda.synchronize()
    for p0, p, g, m0, m in zip(ps, p32, gs, ms, m32):
        want_m = m0 * np.float32(0.9)
        want_m += g.float()
        assert torch.equal(m, want_m)
        u = g.double() + 0.9 * m.double() if nesterov else m.double()
        o = om.newton_schulz(u)
        err = _scheme_error(u, o)
        eta = 0.02 * ops.muon_lr_factor(*p.shape)
        want = p0.double() * (1 - 0.02 * 0.1) - eta * o
        size = torch.linalg.norm(p0.double()) + eta * torch.linalg.norm(o)
        got = torch.linalg.norm(p.double() - want)
        assert got <= eta * err * torch.linalg.norm(o) + 3 * 2.0 ** -24 * size
    for rounding in ("rn", "sr"):
        pb, mb = [p.clone() for p in ps], [m.clone() for m in ms]
        ops.muon_step(pb, gs, mb, bases, rounding=rounding, **hp)
        torch.cuda.synchronize()
        for p, y, base, m, m2 in zip(pb, p32, bases, mb, m32):
            want = oracle.gemm_round(to_host(y), rounding, 11, 3, base)
            assert_bits_equal(to_host(p).reshape(-1), want.reshape(-1), rounding)
            assert torch.equal(m, m2)


def test_muon_step_options():
    announce("muon_step options")
    shape = (48, 96)
    (p,), (g,), (m,) = _state([shape], torch.float32, torch.float32)
    q, n = p.clone(), m.clone()
    ops.muon_step([q], [g], [n], [0], lr=0.1, adjust_lr="match_rms_adamw", step=1, seed=0)
    o = om.newton_schulz(g.double() + 0.95 * (0.95 * m.double() + g.double()))
    err = 2 * om.relative(om.newton_schulz_f16(g.double() + 0.95 * n.double()), o) + SUMS
    eta = 0.1 * 0.2 * 96 ** 0.5
    # (u here is formed in 64 bits: three f32 roundings of it, in directions
    # that the orthogonalisation multiplies by up to 3.4445**5 = 485)
    err += 485 * 3 * 2.0 ** -24
    d = torch.linalg.norm(q.double() - (p.double() - eta * o))
    assert d <= eta * err * torch.linalg.norm(o) + 2.0 ** -22 * torch.linalg.norm(p.double())
    # two lists of one shape but other types go through together, empty ones too
    a = [p.clone(), p.bfloat16(), torch.empty(0, 4, device="cuda")]
    ms = [m.clone(), m.clone(), torch.empty(0, 4, device="cuda")]
    gs = [g, g.clone(), torch.empty(0, 4, device="cuda")]
    ops.muon_step(a, gs, ms, [0, 0, 0], lr=0.1, adjust_lr="match_rms_adamw", step=1, seed=0)
    assert torch.equal(a[0], q) and torch.equal(ms[0], n) and torch.equal(ms[1], n)


def test_shared_memory_is_refused():
    announce("muon overlap")
    p = torch.ones(8, 8, device="cuda")
    with pytest.raises(ValueError, match="share memory"):
        ops.muon_step([p], [p], [torch.zeros(8, 8, device="cuda")], [0], lr=0.1, step=1, seed=0)
    with pytest.raises(ValueError, match="share memory"):
        raw = torch.zeros(8 * 8 * 2, dtype=torch.bfloat16, device="cuda")
        ops.newton_schulz(raw.view(torch.float32).view(8, 8), out=raw[:64].view(8, 8))
    with pytest.raises(ValueError, match="contiguous"):
        ops.newton_schulz(torch.ones(8, 8, device="cuda").t()[:, ::2])
    assert bool((p == 1).all())


def test_optimizer_against_steps():
    """MuonSR's step is muon_step with its positions and counts; a saved and
    loaded optimizer goes on as the first would."""
    announce("MuonSR")
    shapes = [(40, 70), (70, 40), (40, 70)]
    ps, gs, _ = _state(shapes, torch.bfloat16, torch.bfloat16, seed=3)
    params = [torch.nn.Parameter(p.clone()) for p in ps]
    opt = MuonSR(params, lr=0.02, weight_decay=0.1, seed=9, base_offset=17)
    ms = [torch.zeros(s, device="cuda") for s in shapes]
    bases = [17, 17 + 2800, 17 + 5600]
    for t in (1, 2, 3):
        for p, g in zip(params, gs):
            p.grad = g * t
        opt.step()
        ops.muon_step(ps, [g * t for g in gs], ms, bases, lr=0.02, weight_decay=0.1, step=t,
                      seed=9)
        for p, q in zip(params, ps):
            assert torch.equal(p.detach().view(torch.int16), q.view(torch.int16)), t
    sd = opt.state_dict()
    fresh = [torch.nn.Parameter(p.detach().clone()) for p in params]
    two = MuonSR(fresh, lr=1.0, seed=1, base_offset=17)
    two.load_state_dict(sd)
    for p, q, g in zip(params, fresh, gs):
        p.grad = q.grad = g
    opt.step()
    two.step()
    for p, q in zip(params, fresh):
        assert torch.equal(p.detach().view(torch.int16), q.detach().view(torch.int16))


def test_captured_step():
    """The Muon step captured into a graph and replayed, each replay checked
    against the eager steps (the captured step repeats its number)."""
    announce("muon capture")
    shapes = [(70, 130), (256, 256), (70, 130)]
    ps, gs, ms = _state(shapes, torch.bfloat16, torch.bfloat16, seed=5)
    ws = torch.empty(ops.muon_workspace_bytes(shapes), dtype=torch.uint8, device="cuda")

    def once(p, m):
        ops.muon_step(p, gs, m, [0, 10000, 90000], lr=0.02, weight_decay=0.1, step=2, seed=4,
                      workspace=ws)

    pe, me = [p.clone() for p in ps], [m.clone() for m in ms]
    want = []
    for _ in range(3):
        once(pe, me)
        torch.cuda.synchronize()
        want.append(([to_host(p) for p in pe], [to_host(m) for m in me]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        once(ps, ms)
    for r in range(3):
        graph.replay()
        torch.randn(1 << 18, device="cuda").sum().item()
        torch.cuda.synchronize()
        for got, ref in zip((ps, ms), want[r]):
            for a, b in zip(got, ref):
                assert np.array_equal(to_host(a), b), r


def test_training_step_with_int8_products():
    """A two-layer network with bf16 weights: its products in int8 with
    stochastic gradients, its matrices updated by MuonSR and its gain by
    AdamWSR, twice with the same keys. Both runs end in the same bits, every
    weight moves, and the gradients are near those of the same network in
    f32 (each product's int8 error is below (sa/2) sum|b| + (sb/2) sum|a|,
    with one step instead of half for the stochastic operand; checked for the
    last layer, whose inputs both networks share)."""
    announce("int8 + muon training")

    def train():
        gen = torch.Generator(device="cuda")
        gen.manual_seed(1)
        w1 = torch.nn.Parameter((torch.randn(96, 64, generator=gen, device="cuda") * 0.1).bfloat16())
        w2 = torch.nn.Parameter((torch.randn(32, 96, generator=gen, device="cuda") * 0.1).bfloat16())
        gain = torch.nn.Parameter(torch.ones(64, device="cuda", dtype=torch.bfloat16))
        start = [p.detach().clone() for p in (w1, w2, gain)]
        muon = MuonSR([w1, w2], lr=0.02, seed=3, base_offset=64)
        adamw = AdamWSR([gain], lr=1e-2, seed=3)
        x = torch.randn(50, 64, generator=gen, device="cuda").bfloat16()
        y = torch.randn(50, 32, generator=gen, device="cuda").bfloat16()
        for t in range(1, 4):
            h = linear_i8(x * gain, w1, seed=5, step=t, base_index=0)
            a = torch.relu(h)
            a.retain_grad()
            z = linear_i8(a, w2, seed=5, step=t, base_index=50 * 96)
            z.retain_grad()
            (z - y).float().square().mean().backward()
            dz, av = z.grad.double(), a.detach().double()
            exact = dz.T @ av
            sd = dz.abs().amax(0)[:, None] / 127
            sa = av.abs().amax(0)[None, :] / 127
            bound = sd * av.abs().sum(0)[None, :] + sa / 2 * dz.abs().sum(0)[:, None] + 50 * sd * sa / 2
            err = (w2.grad.double() - exact).abs()
            assert bool((err <= 1.001 * (bound + 2.0 ** -8 * (exact.abs() + bound))).all())
            muon.step()
            adamw.step()
            for p in (w1, w2, gain):
                assert torch.isfinite(p.grad).all()
                p.grad = None
        for p, s in zip((w1, w2, gain), start):
            assert bool((p.detach() != s).any())
        return [to_host(p) for p in (w1, w2, gain)]

    one, two = train(), train()
    for a, b in zip(one, two):
        assert np.array_equal(a, b)


def test_long_mixed_list():
    """More matrices than one launch takes, large and small ones of both
    orientations mixed, ragged widths: each ends as it does alone."""
    announce("muon mixed list")
    shapes = [(130 + 2 * (i % 7), 140 + 3 * (i % 5)) for i in range(37)]
    shapes[3:3] = [(20 + i, 40 + 5 * (i % 3)) for i in range(35)]
    shapes[50] = (700, 260)
    shapes[20] = (260, 900)
    ps, gs, ms = _state(shapes, torch.bfloat16, torch.float32, seed=7)
    bases = [17 + 1000 * i for i in range(len(shapes))]
    hp = dict(lr=0.02, weight_decay=0.1, step=5, seed=2)
    pa, ma = [p.clone() for p in ps], [m.clone() for m in ms]
    ops.muon_step(pa, gs, ma, bases, **hp)
    for i in range(len(shapes)):
        p, m = ps[i].clone(), ms[i].clone()
        ops.muon_step([p], [gs[i]], [m], [bases[i]], **hp)
        assert torch.equal(p.view(torch.int16), pa[i].view(torch.int16)), (i, shapes[i])
        assert torch.equal(m, ma[i]), (i, shapes[i])


def test_unaligned_matrices():
    """Weights, gradients and momenta that start on no vector boundary."""
    announce("muon unaligned")
    for shape in ((40, 64), (200, 264), (264, 200)):
        for pt in (torch.bfloat16, torch.float32):
            (p,), (g,), (m,) = _state([shape], pt, torch.bfloat16, seed=11)
            a, b = p.clone(), m.clone()
            ops.muon_step([a], [g], [b], [3], lr=0.02, step=1, seed=5)

            def off(t):
                store = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
                store[1:].copy_(t.reshape(-1))
                return store[1:].view(t.shape)

            q, h, n = off(p), off(g), off(m)
            ops.muon_step([q], [h], [n], [3], lr=0.02, step=1, seed=5)
            assert torch.equal(q, a) and torch.equal(n, b), (shape, pt)


def test_two_streams_at_once():
    """Two optimizers' steps on two streams at once, each with its workspace."""
    announce("muon two streams")
    shapes = [(300, 500), (500, 300), (64, 64)]
    start = [_state(shapes, torch.bfloat16, torch.bfloat16, seed=20 + k) for k in range(2)]

    def make(k):
        params = [torch.nn.Parameter(p.clone()) for p in start[k][0]]
        for p, g in zip(params, start[k][1]):
            p.grad = g.clone()
        return params, MuonSR(params, lr=0.02, seed=k)

    want = []
    for k in range(2):
        params, opt = make(k)
        for _ in range(4):
            opt.step()
        want.append([to_host(p) for p in params])
    streams = [torch.cuda.Stream() for _ in range(2)]
    made = [make(k) for k in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for (params, opt), st in zip(made, streams):
            with torch.cuda.stream(st):
                opt.step()
    torch.cuda.synchronize()
    for k in range(2):
        for p, v in zip(made[k][0], want[k]):
            assert np.array_equal(to_host(p), v)


def test_optimizer_over_two_types():
    """Matrices of two types in one group of the optimizer, whose own lists
    need more workspace than the list of both: as a step for each type."""
    announce("MuonSR two types")
    shapes = [(1024, 1040), (40, 1040)] * 20
    dtypes = [torch.bfloat16, torch.float32] * 20
    ps, gs, ms = [], [], []
    for i in range(2):
        p, g, m = _state(shapes[i::2], dtypes[i], dtypes[i], seed=i)
        ps.append(p), gs.append(g), ms.append([torch.zeros_like(x) for x in m])
    params = [torch.nn.Parameter(ps[k % 2][k // 2].clone()) for k in range(40)]
    opt = MuonSR(params, lr=0.02, seed=4)
    for k, p in enumerate(params):
        p.grad = gs[k % 2][k // 2]
    opt.step()
    bases = [opt.base_index(p) for p in params]
    for i in range(2):
        ops.muon_step(ps[i], gs[i], ms[i], bases[i::2], lr=0.02, weight_decay=0.1, step=1, seed=4)
        for p, q, m in zip(params[i::2], ps[i], ms[i]):
            assert torch.equal(p.detach(), q)
            assert torch.equal(opt.state[p]["momentum_buffer"], m)


def test_captured_optimizer():
    """MuonSR's step in two graphs, replayed in turn, against eager steps (a
    captured step repeats its number); a first step is not captured."""
    announce("MuonSR capture")
    shapes = [(300, 200), (64, 64), (130, 260)]
    ps, gs, _ = _state(shapes, torch.bfloat16, torch.bfloat16, seed=6)
    params = [torch.nn.Parameter(p.clone()) for p in ps]
    opt = MuonSR(params, lr=0.02, seed=4)
    for p, g in zip(params, gs):
        p.grad = g
    opt.step()   # step 1; the graphs hold steps 2 and 3
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph in graphs:
        with torch.cuda.graph(graph):
            opt.step()
    ms = [torch.zeros(s, device="cuda") for s in shapes]
    bases = [opt.base_index(p) for p in params]
    for step in (1, 2, 3, 2, 3, 3):
        ops.muon_step(ps, gs, ms, bases, lr=0.02, weight_decay=0.1, step=step, seed=4)
        if step > 1:
            graphs[step - 2].replay()
            torch.randn(1 << 18, device="cuda").sum().item()
        torch.cuda.synchronize()
        for p, q in zip(params, ps):
            assert torch.equal(p.detach().view(torch.int16), q.view(torch.int16)), step


def test_workspace_may_not_be_the_data():
    announce("muon workspace overlap")
    g = torch.ones(200, 300, dtype=torch.bfloat16, device="cuda")
    need = ops.muon_workspace_bytes([(200, 300)])
    raw = torch.zeros(need + 2 * g.numel(), dtype=torch.uint8, device="cuda")
    out = raw[need:].view(torch.bfloat16).view(200, 300)
    with pytest.raises(ValueError, match="share memory"):
        ops.newton_schulz(g, out=out, workspace=raw)
    with pytest.raises(ValueError, match="contiguous"):
        ops.newton_schulz(g, workspace=torch.zeros(2 * need, dtype=torch.uint8, device="cuda")[::2])
    with pytest.raises(ValueError, match="share memory"):
        ops.muon_step([g], [out], [torch.zeros(200, 300, device="cuda")], [0], lr=0.1, step=1,
                      seed=0, workspace=raw)
    assert bool((g == 1).all()) and bool((out == 0).all())
    ops.newton_schulz(g, out=out, workspace=raw[:need])
    assert torch.equal(out, ops.newton_schulz(g))


def test_refused_list_changes_nothing():
    """A matrix that only a later type's list would refuse: no matrix of the
    types before it has moved, so a step taken again is not taken twice."""
    announce("muon refusal before the first launch")
    (p,), (g,), (m,) = _state([(40, 70)], torch.bfloat16, torch.bfloat16)
    long = [torch.zeros(1, 2 ** 20 + 1, device="cuda") for _ in range(3)]
    q, n = p.clone(), m.clone()
    with pytest.raises((ValueError, ops.AsrError), match="2\\*\\*20"):
        ops.muon_step([q, long[0]], [g, long[1]], [n, long[2]], [0, 0], lr=0.1, step=1, seed=0)
    torch.cuda.synchronize()
    assert torch.equal(q, p) and torch.equal(n, m)


def _newton_schulz_bf16(u):
    """The scheme that torch.optim.Muon's documentation names: products of bf16
    matrices (sums in binary64 here, every result rounded to bf16)."""
    def r(x):
        return x.to(torch.bfloat16).double()

    a, b, c = om.COEFFICIENTS
    x = r(u if u.shape[0] <= u.shape[1] else u.T)
    x = r(x / torch.linalg.norm(x))
    for _ in range(5):
        gram = r(x @ x.T)
        x = r(a * x + r(b * gram + c * r(gram @ gram)) @ x)
    return x if u.shape[0] <= u.shape[1] else x.T


@pytest.mark.parametrize("nesterov", [True, False], ids=["nesterov", "plain"])
@pytest.mark.parametrize("adjust", [None, "match_rms_adamw"])
def test_against_torch_muon(adjust, nesterov):
    """Three steps of torch.optim.Muon (on the CPU) and of MuonSR on f32 weights,
    then a fourth of a MuonSR that was given torch's state: apart by twice what
    the bf16 scheme and this one are off, a step (a wrong scale of the momentum
    would turn u: the gradients of the steps are independent)."""
    announce("MuonSR against torch.optim.Muon", adjust, nesterov)
    shapes = [(48, 96), (150, 200), (200, 70)]
    kw = dict(lr=0.05, weight_decay=0.2, momentum=0.9, nesterov=nesterov, adjust_lr_fn=adjust)
    start = [_matrix("normal", *s, seed=i, dtype=torch.float32) * 20 for i, s in enumerate(shapes)]
    theirs = [torch.nn.Parameter(p.cpu()) for p in start]
    mine = [torch.nn.Parameter(p.clone()) for p in start]
    opt_t, opt_m = torch.optim.Muon(theirs, **kw), MuonSR(mine, **kw)
    limit, m64 = [0.0] * 3, [torch.zeros(s, dtype=torch.float64, device="cuda") for s in shapes]

    def one(params, opt, t):
        for i, (p, q) in enumerate(zip(theirs, params)):
            g = _matrix("normal", *shapes[i], seed=10 * t + i, dtype=torch.float32)
            p.grad, q.grad = g.cpu(), g
            m64[i] = 0.9 * m64[i] + g.double()
            u = g.double() + 0.9 * m64[i] if nesterov else m64[i]
            o = om.newton_schulz(u)
            off = om.relative(_newton_schulz_bf16(u), o) + om.relative(om.newton_schulz_f16(u), o) + SUMS
            eta = 0.05 * ops.muon_lr_factor(*shapes[i], adjust or "original")
            limit[i] += 2 * off * eta * torch.linalg.norm(o).item()
        opt_t.step()
        opt.step()
        for i, (p, q) in enumerate(zip(theirs, params)):
            d = torch.linalg.norm(p.detach().double() - q.detach().double().cpu()).item()
            assert d <= limit[i], (t, i)

    for t in (1, 2, 3):
        one(mine, opt_m, t)
    moved = [torch.nn.Parameter(p.detach().cuda()) for p in theirs]
    opt = MuonSR(moved, lr=1.0)
    opt.load_state_dict(opt_t.state_dict())
    assert opt.param_groups[0]["lr"] == 0.05
    limit = [0.0] * 3
    one(moved, opt, 4)


def test_positions_past_the_last():
    """Global positions wrap modulo 2**64."""
    announce("muon positions wrap")
    shapes = [(40, 70), (200, 264), (130, 515)]
    ps, gs, ms = _state(shapes, torch.bfloat16, torch.bfloat16, seed=31)
    bases = [2 ** 64 - 1000, 2 ** 64 - 4, 2 ** 64 - 3]
    p32, m32 = [p.float() for p in ps], [m.clone() for m in ms]
    hp = dict(lr=0.02, weight_decay=0.1, step=2 ** 32 - 1, seed=2 ** 32 - 1)
    ops.muon_step(p32, gs, m32, bases, **hp)
    ops.muon_step(ps, gs, ms, bases, **hp)
    torch.cuda.synchronize()
    for p, y, base in zip(ps, p32, bases):
        want = oracle.gemm_round(to_host(y), "sr", 2 ** 32 - 1, 2 ** 32 - 1, base)
        assert_bits_equal(to_host(p).reshape(-1), want.reshape(-1), base)
