"""Refusals of the Newton-Schulz and Muon entry points, and MuonSR's host side
(CPU only; no call here launches a kernel)."""

import ctypes

import pytest
import torch

from adamw_optimizer_stochastic_amd import MuonSR, _abi, _build, ops

NS = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module", autouse=True)
def built():
    if not _build.is_built():
        _build.build()


def _status(fn, *args):
    try:
        fn(*args)
    except _abi.AsrError as e:
        return e.status
    return _abi.ASR_OK


def test_newton_schulz_argument_errors():
    E = _abi
    need = E.asr_newton_schulz_workspace_bytes(1, 400, 600)

    def f(g=(0x1000,), out=(0x80000,), rows=400, cols=600, dtype=E.ASR_BF16, steps=5, coeffs=NS,
          eps=1e-7, ws=0x100000, ws_bytes=need):
        return _status(E.asr_newton_schulz, g, out, rows, cols, dtype, steps, *coeffs, eps, ws,
                       ws_bytes, None)

    assert f(rows=-1) == E.ASR_EINVAL
    assert f(cols=2 ** 20 + 1) == E.ASR_EINVAL
    assert f(dtype=7) == E.ASR_EDTYPE
    assert f(steps=0) == E.ASR_EINVAL
    assert f(steps=65) == E.ASR_EINVAL
    assert f(eps=-1.0) == E.ASR_EINVAL
    assert f(eps=float("nan")) == E.ASR_EINVAL
    # singular values would leave the range the f16 operands are scaled for
    assert f(coeffs=(8.0, -20.0, 14.0)) == E.ASR_EINVAL
    assert f(coeffs=(float("nan"), 0.0, 0.0)) == E.ASR_EINVAL
    assert f(coeffs=(1.0, 5.0, 0.0)) == E.ASR_EINVAL
    assert f(g=(0,)) == E.ASR_EINVAL
    assert f(out=(0,)) == E.ASR_EINVAL
    assert f(g=(0x1001,)) == E.ASR_EALIGN
    assert f(dtype=E.ASR_F32, g=(0x1002,)) == E.ASR_EALIGN
    assert f(out=(0x80001,)) == E.ASR_EALIGN
    assert f(ws=0) == E.ASR_EWORKSPACE
    assert f(ws=0x100080) == E.ASR_EWORKSPACE
    assert f(ws_bytes=need - 1) == E.ASR_EWORKSPACE
    assert f(g=(), out=()) == E.ASR_OK
    assert f(rows=0, g=(0,), out=(0,), ws=0, ws_bytes=0) == E.ASR_OK


def test_accepted_coefficients():
    """The usual choices pass the range check (the missing workspace is what
    stops the call)."""
    E = _abi
    for c in (NS, (1.5, -0.5, 0.0), (1.875, -1.25, 0.375), (2.0, -1.5, 0.5)):
        got = _status(E.asr_newton_schulz, (0x1000,), (0x8000,), 300, 300, E.ASR_BF16, 5, *c, 1e-7, 0,
                      0, None)
        assert got == E.ASR_EWORKSPACE, c


def test_workspace_bytes():
    f = _abi.asr_newton_schulz_workspace_bytes
    assert f(0, 800, 800) == 0 and f(1, 0, 8) == 0 and f(1, -1, 8) == 0
    one = f(1, 200, 300)
    assert one >= 8 * 200 * 300 + 4 * 200 * 200
    assert f(1, 300, 200) >= 8 * 200 * 300 + 4 * 200 * 200
    assert f(3, 200, 300) == 3 * one
    assert f(32, 200, 300) == f(500, 200, 300) == 32 * one   # at most 32 at a time
    big = f(1, 8192, 28672)
    assert f(9, 8192, 28672) == max(1, (4 << 30) // big) * big
    # a matrix that one workgroup holds needs none
    assert f(7, 128, 128) == f(7, 64, 512) == f(7, 1, 1) == 0
    # a list of several shapes: groups of it share the workspace, so more
    # matrices never need less, and small ones add nothing
    w = ops.muon_workspace_bytes
    assert w([(200, 300)]) == one and w([(200, 300), (64, 64), (0, 5)]) == one
    assert w([(200, 300), (300, 200)]) == one + f(1, 300, 200)
    assert w([]) == 0 and w([(64, 64)] * 40) == 0
    assert w([(200, 300)] * 40) == 32 * one


def test_muon_argument_errors():
    E = _abi
    need = E.asr_newton_schulz_workspace_bytes(1, 400, 600)
    good = (0x1000, 0x80000, 0x100000, 400, 600, 0, 1.0)
    assert ctypes.sizeof(E.AsrMuonTensor) == 56

    def f(t=good, pt=E.ASR_BF16, gt=E.ASR_BF16, lr=0.1, mu=0.9, wd=0.1, steps=5, coeffs=NS,
          eps=1e-7, step=1, rounding=E.ASR_ROUND_SR, ws=0x1000000, ws_bytes=need):
        return _status(E.asr_muon_step, E.muon_array([t]), 1, pt, gt, lr, mu, 1, wd, steps,
                       coeffs, eps, step, 0, rounding, ws, ws_bytes, None)

    def but(i, v):
        return tuple(v if j == i else x for j, x in enumerate(good))

    assert f(t=but(3, -1)) == E.ASR_EINVAL
    assert f(t=but(4, 2 ** 20 + 1)) == E.ASR_EINVAL
    assert f(pt=4) == E.ASR_EDTYPE
    assert f(gt=4) == E.ASR_EDTYPE
    for bad in (-0.1, float("inf"), float("nan")):
        assert f(lr=bad) == E.ASR_EINVAL
        assert f(wd=bad) == E.ASR_EINVAL
        assert f(t=but(6, bad)) == E.ASR_EINVAL
        assert f(mu=bad) == E.ASR_EINVAL
    assert f(mu=1.0) == E.ASR_EINVAL
    assert f(step=0) == E.ASR_EINVAL
    assert f(step=2 ** 32) == E.ASR_EINVAL
    assert f(rounding=2) == E.ASR_EINVAL
    assert f(steps=0) == E.ASR_EINVAL
    assert f(eps=-1.0) == E.ASR_EINVAL
    for i in range(3):
        assert f(t=but(i, 0)) == E.ASR_EINVAL
    assert f(t=but(0, 0x1001)) == E.ASR_EALIGN
    assert f(t=but(2, 0x100002)) == E.ASR_EALIGN
    assert f(ws=0) == E.ASR_EWORKSPACE
    assert f(ws=0x1000080) == E.ASR_EWORKSPACE
    assert f(ws_bytes=need - 1) == E.ASR_EWORKSPACE
    assert f(t=but(4, 0), ws=0, ws_bytes=0) == E.ASR_OK


def test_binding_refusals():
    x = torch.zeros(4, 6)
    with pytest.raises(ValueError, match="GPU"):
        ops.newton_schulz(x)
    with pytest.raises(ValueError, match="three"):
        ops.newton_schulz(x, coefficients=(1.0, 2.0))
    with pytest.raises(ValueError, match="GPU"):
        ops.muon_step([x], [x], [x], [0], lr=0.1, step=1, seed=0)
    with pytest.raises(ValueError, match="length"):
        ops.muon_step([x], [x], [], [0], lr=0.1, step=1, seed=0)
    with pytest.raises(ValueError, match="adjust_lr"):
        ops.muon_step([], [], [], [], lr=0.1, step=1, seed=0, adjust_lr="none")
    with pytest.raises(ValueError, match="step"):
        ops.muon_step([], [], [], [], lr=0.1, step=0, seed=0)
    ops.muon_step([], [], [], [], lr=0.1, step=1, seed=0)


def test_lr_factor():
    f = ops.muon_lr_factor
    assert f(100, 400) == 1.0 and f(400, 100) == 2.0
    assert f(100, 400, "match_rms_adamw") == f(400, 100, "match_rms_adamw") == 0.2 * 20


def _param(*shape, dtype=torch.float32):
    return torch.nn.Parameter(torch.zeros(shape, dtype=dtype))


def test_optimizer_refusals():
    for kw in (dict(lr=-1.0), dict(weight_decay=-1.0), dict(momentum=1.0), dict(eps=-1.0),
               dict(ns_steps=0), dict(rounding="up"), dict(seed=-1), dict(adjust_lr_fn="x"),
               dict(base_offset=-1), dict(ns_coefficients=(1.0,))):
        with pytest.raises(ValueError):
            MuonSR([_param(4, 4)], **kw)
    with pytest.raises(NotImplementedError):
        MuonSR([_param(4, 4)], lr=torch.tensor(0.1))
    with pytest.raises(ValueError, match="2-D"):
        MuonSR([_param(4)])
    with pytest.raises(NotImplementedError):
        MuonSR([_param(4, 4, dtype=torch.float64)])


def test_optimizer_positions_and_state():
    a, b, c = _param(3, 4), _param(5, 2, dtype=torch.bfloat16), _param(2, 2)
    opt = MuonSR([a, b], seed=7, base_offset=100)
    opt.add_param_group(dict(params=[c], lr=0.5))
    assert [opt.base_index(p) for p in (a, b, c)] == [100, 112, 122]
    assert opt.param_groups[0]["adjust_lr_fn"] == "original"
    for p in (a, b):
        opt._init_state(p)
    opt.state[b]["momentum_buffer"].fill_(1.0009765625)   # not a bf16 number
    opt.state[b]["step"].fill_(2 ** 25 + 1)               # not a float32 number
    sd = opt.state_dict()
    other = MuonSR([_param(3, 4), _param(5, 2, dtype=torch.bfloat16)], seed=1)
    other.add_param_group(dict(params=[_param(2, 2)]))
    other.load_state_dict(sd)
    p = other.param_groups[0]["params"][1]
    assert other.seed == 7 and int(other.state[p]["step"]) == 2 ** 25 + 1
    assert other.state[p]["momentum_buffer"].dtype == torch.float32
    assert bool((other.state[p]["momentum_buffer"] == 1.0009765625).all())
    assert other.param_groups[1]["lr"] == 0.5
    opt.step()   # no gradients: nothing to do


def test_optimizer_step_leaves_workspaces_to_each_call(monkeypatch):
    """Types of one group go through the products apart, and the most that one
    type's list needs can be more than what the whole list needs (its groups of
    32 mix large and small matrices): a workspace sized for the whole list is
    too small."""
    big, low = [(1024, 1040)] * 20, [(40, 1040)] * 20
    mixed = [s for pair in zip(big, low) for s in pair]
    assert ops.muon_workspace_bytes(big) > ops.muon_workspace_bytes(mixed)
    calls = []
    monkeypatch.setattr(ops, "muon_step", lambda *a, **kw: calls.append((a, kw)))
    params = [_param(4, 6), _param(4, 6, dtype=torch.bfloat16), _param(4, 6)]
    opt = MuonSR(params, seed=3)
    for p in params[:2]:
        p.grad = torch.ones_like(p)
    opt.step()
    (args, kw), = calls
    assert [p.dtype for p in args[0]] == [torch.float32, torch.bfloat16]
    assert kw.get("workspace") is None and kw["step"] == 1 and args[3] == [0, 24]


def test_first_step_is_not_captured(monkeypatch):
    """Its momentum of zeros would be part of the graph."""
    class OnGpu:
        is_cuda, shape, device = True, (4, 6), "cpu"
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    opt = MuonSR([_param(4, 6)])
    with pytest.raises(RuntimeError, match="before capturing"):
        opt._init_state(OnGpu())


BAD_OPTIONS = (dict(lr=-1.0), dict(lr=float("inf")), dict(weight_decay=-1.0),
               dict(weight_decay=float("nan")), dict(momentum=1.0), dict(momentum=2.0),
               dict(eps=-1.0), dict(eps=float("inf")), dict(ns_steps=0), dict(ns_steps=65),
               dict(rounding="xx"), dict(adjust_lr_fn="x"), dict(ns_coefficients=(1.0,)))


@pytest.mark.parametrize("kw", BAD_OPTIONS, ids=str)
def test_options_of_a_group_are_checked(kw):
    """As the constructor's are; the refused group leaves nothing behind."""
    a = _param(4, 6)
    opt = MuonSR([a], base_offset=5)
    with pytest.raises(ValueError):
        MuonSR([_param(4, 6)], **kw)
    with pytest.raises(ValueError):
        MuonSR([dict(params=[_param(4, 6)], **kw)])
    with pytest.raises(ValueError):
        opt.add_param_group(dict(params=[_param(4, 6)], **kw))
    assert len(opt.param_groups) == 1 and len(opt._base_index) == 1 and opt._next_index == 29


def test_refused_groups_leave_nothing_behind():
    opt = MuonSR([_param(4, 6)])
    tensor_lr, float_steps = dict(lr=torch.tensor(0.1)), dict(ns_steps=2.5)
    for params, kw, error in (([_param(4)], {}, ValueError),
                              ([_param(3, 3), _param(2, 2, 2)], {}, ValueError),
                              ([_param(0, 2 ** 20 + 1)], {}, ValueError),
                              ([_param(3, 3, dtype=torch.float64)], {}, NotImplementedError),
                              ([_param(3, 3)], tensor_lr, NotImplementedError),
                              ([_param(3, 3)], float_steps, TypeError)):
        with pytest.raises(error):
            opt.add_param_group(dict(params=params, **kw))
        assert len(opt.param_groups) == 1 and len(opt._base_index) == 1
    b = _param(2, 5)
    opt.add_param_group(dict(params=(p for p in [b]), adjust_lr_fn=None, ns_coefficients=[2, -1.5, 0.5]))
    assert opt.base_index(b) == 24   # the refused ones took no positions
    assert opt.param_groups[1]["adjust_lr_fn"] == "original"
    assert opt.param_groups[1]["ns_coefficients"] == (2.0, -1.5, 0.5)


def test_state_of_torch_muon_is_taken():
    """Its buffer is 1 - momentum times this one's; it has no step count and no
    rounding."""
    a, b = _param(3, 4), _param(5, 2)
    theirs = torch.optim.Muon([dict(params=[a], momentum=0.5), dict(params=[b], lr=0.25)])
    for p in (a, b):
        p.grad = torch.full_like(p, 3.0)
    theirs.step()
    mine = [_param(3, 4), _param(5, 2, dtype=torch.bfloat16)]
    opt = MuonSR([dict(params=[p]) for p in mine], seed=3, rounding="rn")
    opt.load_state_dict(theirs.state_dict())
    for p in mine:   # one step's sum is its gradient; two factors and a quotient rounded to binary32
        st = opt.state[p]
        assert st["momentum_buffer"].dtype == torch.float32 and int(st["step"]) == 0
        assert torch.allclose(st["momentum_buffer"], torch.full((), 3.0), rtol=2.0 ** -21)
    one, two = opt.param_groups
    assert (one["momentum"], two["momentum"], two["lr"]) == (0.5, 0.95, 0.25)
    assert one["adjust_lr_fn"] == "original" and one["rounding"] == "rn" and opt.seed == 3


def test_state_that_does_not_fit_changes_nothing():
    p = _param(3, 4)
    opt = MuonSR([p], lr=0.5, seed=3)
    opt._init_state(p)
    opt.state[p]["momentum_buffer"].fill_(2.0)
    opt.state[p]["step"].fill_(4)
    good = opt.state_dict()

    def but(state=None, **group):
        sd = dict(good, param_groups=[dict(good["param_groups"][0], **group)])
        return sd if state is None else dict(sd, state={0: state})

    for sd, match in ((but(dict(step=1, exp_avg=torch.ones(3, 4))), "momentum_buffer"),
                      (but(dict(step=1, momentum_buffer=torch.ones(3, 5))), "momentum_buffer"),
                      (but(dict(step=1.5, momentum_buffer=torch.ones(3, 4))), "step count"),
                      (but(lr=-1.0), "learning rate"), (but(rounding="xx"), "rounding")):
        with pytest.raises(ValueError, match=match):
            opt.load_state_dict(sd)
        assert opt.param_groups[0]["lr"] == 0.5 and int(opt.state[p]["step"]) == 4
        assert bool((opt.state[p]["momentum_buffer"] == 2.0).all())
    with pytest.raises(ValueError, match="parameter group"):
        opt.load_state_dict(dict(good, param_groups=good["param_groups"] * 2))
    opt.load_state_dict(good)
    assert int(opt.state[p]["step"]) == 4


def test_refused_gradient_moves_nothing(monkeypatch):
    """A gradient of a later group that the step refuses is found before the first
    group moves."""
    calls = []
    monkeypatch.setattr(ops, "muon_step", lambda *a, **kw: calls.append(a))
    a, b = _param(4, 6), _param(4, 6)
    opt = MuonSR([dict(params=[a]), dict(params=[b], lr=0.5)])
    a.grad = torch.ones(4, 6)
    for bad in (torch.ones(6, 4).t(), torch.eye(4, 6).to_sparse()):
        b.grad = bad
        with pytest.raises(NotImplementedError):
            opt.step()
        assert not calls and int(opt.state[a].get("step", 0)) == 0
    b.grad = torch.ones(4, 6)
    opt.step()
    assert len(calls) == 2 and int(opt.state[a]["step"]) == int(opt.state[b]["step"]) == 1
