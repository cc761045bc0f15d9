"""Gradients whose saved tensors autograd hands back in another layout or computes
again: offload to host memory, copies, rows further apart, checkpoints. The
kernels read the same values, so every gradient has the bits of the pass without."""

import contextlib

import pytest
import torch

from adamw_optimizer_stochastic_amd import embedding, layer_norm, linear_i8, silu_mul
from _gpu_util import announce, gpu, require_gpu

pytestmark = gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def _spread(t):
    if not t.dtype.is_floating_point or t.dim() != 2:
        return t
    wide = t.new_full((*t.shape[:-1], 3 * t.shape[-1] + 5), float("nan"))
    wide[..., 1:1 + t.shape[-1]] = t
    return wide[..., 1:1 + t.shape[-1]]


def _columns(t):
    return t.t().contiguous().t() if t.dim() == 2 else t


HOOKS = {"none": contextlib.nullcontext,
         "host": torch.autograd.graph.save_on_cpu,
         "copies": lambda: torch.autograd.graph.saved_tensors_hooks(lambda t: t.clone(), lambda t: t),
         "apart": lambda: torch.autograd.graph.saved_tensors_hooks(lambda t: t, _spread),
         "columns": lambda: torch.autograd.graph.saved_tensors_hooks(lambda t: t, _columns)}


def _same(call, leaves):
    """Gradients of call() by its leaves under every hook, and under a checkpoint."""
    def grads():
        y = call()
        dy = torch.linspace(-1.0, 2.0, y.numel(), device=y.device).view(y.shape).to(y.dtype)
        return torch.autograd.grad(y, leaves, dy)

    want = grads()
    for name, hooks in HOOKS.items():
        announce("hooks", name)
        with hooks():
            got = grads()
        for g, w in zip(got, want):
            assert torch.equal(g, w), name
    announce("checkpoint")
    y = torch.utils.checkpoint.checkpoint(call, use_reentrant=False)
    dy = torch.linspace(-1.0, 2.0, y.numel(), device=y.device).view(y.shape).to(y.dtype)
    for g, w in zip(torch.autograd.grad(y, leaves, dy), want):
        assert torch.equal(g, w)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("form", ["halves", "joint", "joint slice", "contiguous"])
@pytest.mark.parametrize("saved", ["inputs", "i8"])
def test_silu_mul(form, saved, dtype):
    announce("silu_mul kept", form, saved, dtype)
    torch.manual_seed(3)
    x = torch.randn(37, 4 * 141, device="cuda").to(dtype).requires_grad_()

    def call():
        h = x * 1.5
        if form == "halves":
            gate, up = h.chunk(2, -1)
        elif form == "joint":
            gate, up = h, None
        elif form == "joint slice":
            gate, up = h[:, 3:3 + 2 * 141], None
        else:
            gate, up = (t.contiguous() for t in h.chunk(2, -1))
        return silu_mul(gate, up, saved=saved)

    _same(call, [x])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", [141, 9001])
@pytest.mark.parametrize("saved", ["input", "i8"])
def test_layer_norm(saved, cols, dtype):
    announce("layer_norm kept", saved, cols, dtype)
    torch.manual_seed(4)
    x = torch.randn(37, 2 * cols, device="cuda").to(dtype).requires_grad_()
    w, b = (torch.randn(cols, device="cuda").to(dtype).requires_grad_() for _ in range(2))
    _same(lambda: layer_norm((x * 1.5)[:, 3:3 + cols], w * 1.0, b, saved=saved), [x, w, b])


@pytest.mark.parametrize("saved", ["input", "i8"])
def test_linear(saved):
    announce("linear_i8 kept", saved)
    torch.manual_seed(5)
    x = torch.randn(67, 200, device="cuda").bfloat16().requires_grad_()
    w = torch.randn(45, 100, device="cuda").bfloat16().requires_grad_()
    _same(lambda: linear_i8((x * 1.5)[:, 3:103], w * 1.0, seed=1, step=2, saved=saved), [x, w])


@pytest.mark.parametrize("tokens", [200, 5000])
def test_embedding(tokens):
    announce("embedding kept", tokens)
    torch.manual_seed(6)
    ids = torch.randint(0, 37, (tokens // 50, 50), device="cuda")
    w = torch.randn(37, 45, device="cuda").requires_grad_()
    _same(lambda: embedding(ids, w, scale=0.5, padding_idx=3), [w])
