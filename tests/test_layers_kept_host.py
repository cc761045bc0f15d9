"""What the layers' backward passes do with saved tensors that come back from
autograd in another layout (CPU only: the C calls are recorders, no kernel runs)."""

import contextlib

import pytest
import torch

from adamw_optimizer_stochastic_amd import _abi, layers, ops, silu_mul

STORED = (lambda t: t.clone(), lambda t: t)           # as an offload to host memory lays it out
APART = (lambda t: t, lambda t: _spread(t))           # rows further apart than before
COLUMNS = (lambda t: t, lambda t: t.t().contiguous().t() if t.dim() == 2 else t)


def _spread(t):
    wide = t.new_empty((*t.shape[:-1], 3 * t.shape[-1] + 5))
    wide[..., :t.shape[-1]] = t
    return wide[..., :t.shape[-1]]


@pytest.fixture
def calls(monkeypatch):
    """CPU tensors through the Python layer; every C call is recorded instead."""
    made = []

    def record(name):
        monkeypatch.setattr(_abi, name, lambda *args: made.append((name, args)))

    for name in ("asr_silu_mul_forward", "asr_silu_mul_backward"):
        record(name)
    monkeypatch.setattr(layers, "_check_floats", lambda *args: None)
    monkeypatch.setattr(ops, "_on", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(ops, "_stream", lambda device: None)
    return made


def _end(t):
    """One past the last byte of t's storage."""
    return t.untyped_storage().data_ptr() + t.untyped_storage().nbytes()


@pytest.mark.parametrize("hooks", [None, STORED, APART, COLUMNS],
                         ids=["none", "stored", "apart", "columns"])
@pytest.mark.parametrize("joint", [False, True], ids=["halves", "joint"])
def test_silu_mul_walks_the_tensors_it_gets_back(calls, hooks, joint):
    rows, cols = 5, 8
    leaf = torch.randn(rows, 4 * cols, requires_grad=True)
    h = leaf * 2.0
    got = []

    def keep(t):
        got.append(t)
        return t

    pack, unpack = hooks or (lambda t: t, lambda t: t)
    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: keep(unpack(t))):
        y = silu_mul(h[:, :2 * cols]) if joint else silu_mul(h[:, :cols], h[:, cols:2 * cols])
    y.backward(torch.zeros(rows, cols))
    (name, args), = [c for c in calls if c[0] == "asr_silu_mul_backward"]
    g, ld_g, u, ld_u = args[2:6]
    gate, up = got[0], got[-1]
    for p, ld, t, first in ((g, ld_g, gate, 0), (u, ld_u, up, cols if joint else 0)):
        width = 2 * cols if joint else cols
        assert ld >= width
        if t.stride(1) == 1:   # walked where it is: its own address and stride
            assert p == t.data_ptr() + first * 4 and ld == t.stride(0)
            assert p + ((rows - 1) * ld + cols) * 4 <= _end(t)
        else:                  # a copy with contiguous rows
            assert ld == width


def test_silu_mul_refuses_a_tensor_of_another_kind(calls):
    other = {"type": lambda t: t.to(torch.float64), "shape": lambda t: t[:-1],
             "device": lambda t: t.to("meta")}
    for unpack in other.values():
        h = torch.randn(4, 16, requires_grad=True) * 1.0
        with torch.autograd.graph.saved_tensors_hooks(lambda t: t, unpack):
            y = silu_mul(h[:, :8], h[:, 8:])
        with pytest.raises(RuntimeError, match="saved"):
            y.sum().backward()
    assert not [c for c in calls if c[0] == "asr_silu_mul_backward"]


def test_layer_norm_workspace_of_wide_rows():
    """No more of it than the rows themselves are worth: 256 rows of 2**24 columns
    have enough workgroups without sums of their own."""
    from adamw_optimizer_stochastic_amd import _build
    if not _build.is_built():
        _build.build()
    need = _abi.asr_layer_norm_backward_workspace_bytes
    assert need(256, 2 ** 24) == 2 * 2 ** 24 * 4 and need(4, 2 ** 24) == need(256, 2 ** 24)
    for rows, cols in ((64, 131072), (300, 40007), (5000, 16384), (10 ** 6, 8193)):
        strips = -(-cols // 2048)
        assert need(rows, cols) == min(rows, 256, -(-2048 // strips)) * 2 * cols * 4
