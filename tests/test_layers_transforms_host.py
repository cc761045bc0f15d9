"""The layers under forward-mode derivatives and torch.func's transforms, which they
do not have: every call raises, none drops a derivative in silence (CPU only: the C
calls are recorders)."""

import contextlib

import pytest
import torch
import torch.autograd.forward_ad as forward_ad

from adamw_optimizer_stochastic_amd import _abi, embedding, int8, layer_norm, layers, linear_i8, ops, silu_mul

F = torch.float32


@pytest.fixture(autouse=True)
def calls(monkeypatch):
    made = []
    for name in [n for n in dir(_abi) if n.startswith("asr_")]:
        if name.endswith("_workspace_bytes"):
            monkeypatch.setattr(_abi, name, lambda *args: 256)
        elif callable(getattr(_abi, name)):
            monkeypatch.setattr(_abi, name, lambda *args, name=name: made.append(name))
    monkeypatch.setattr(layers, "_check_floats", lambda *args: None)
    monkeypatch.setattr(int8, "_check_operands", lambda *args: None)
    monkeypatch.setattr(ops, "_on", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(ops, "_stream", lambda device: None)
    return made


IDS = torch.tensor([[1, 2, 0]])
# name: (function, its tensors, as (shape, type))
CALLS = {
    "layer_norm": (layer_norm, [((4, 24), F), ((24,), F), ((24,), F)]),
    "layer_norm i8": (lambda *t: layer_norm(*t, saved="i8"), [((4, 24), F), ((24,), F), ((24,), F)]),
    "silu_mul": (silu_mul, [((4, 24), F), ((4, 24), F)]),
    "silu_mul joint": (silu_mul, [((4, 24), F)]),
    "embedding": (lambda w: embedding(IDS, w), [((5, 24), F)]),
    "linear_i8": (linear_i8, [((4, 24), torch.bfloat16), ((8, 24), torch.bfloat16)]),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("grad", [True, False], ids=["grad", "no_grad"])
def test_dual_tensors_are_refused(name, grad):
    call, tensors = CALLS[name]
    for k in range(len(tensors)):
        with forward_ad.dual_level(), torch.set_grad_enabled(grad):
            args = [torch.randn(s).to(t) for s, t in tensors]
            args[k] = forward_ad.make_dual(args[k], torch.ones_like(args[k]))
            with pytest.raises(NotImplementedError, match="forward mode"):
                call(*args)


@pytest.mark.parametrize("name", CALLS)
def test_plain_tensors_beside_dual_ones(name):
    """An open level asks nothing of calls without a tangent."""
    call, tensors = CALLS[name]
    plain = [torch.randn(s).to(t) for s, t in tensors]
    with forward_ad.dual_level():
        y = call(*plain)
        assert not y.requires_grad and forward_ad.unpack_dual(y).tangent is None
        leaves = [t.clone().requires_grad_() for t in plain]
        y = call(*leaves)
        for g, leaf in zip(torch.autograd.grad(y, leaves, torch.zeros_like(y)), leaves):
            assert g.shape == leaf.shape


@pytest.mark.parametrize("name", CALLS)
def test_transforms_are_refused(name, calls):
    call, tensors = CALLS[name]
    args = tuple(torch.randn(s).to(t) for s, t in tensors)
    for run in (lambda: torch.func.jvp(call, args, args),
                lambda: torch.func.grad(lambda *t: call(*t).float().sum())(*args),
                lambda: torch.vmap(call)(*(torch.stack([t, t]) for t in args)),
                lambda: torch.func.jacrev(call)(*args), lambda: torch.func.jacfwd(call)(*args)):
        with pytest.raises((RuntimeError, NotImplementedError)):
            run()
    assert not calls
