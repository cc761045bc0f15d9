"""Saved tensors that come back from autograd's hooks as something else: the
backward passes of layer_norm, embedding and linear_i8 walk them where they are,
or refuse them before a kernel reads their addresses (CPU only: the C calls are
recorders)."""

import contextlib

import pytest
import torch

from adamw_optimizer_stochastic_amd import _abi, embedding, int8, layer_norm, layers, linear_i8, ops

NAMES = ["asr_layer_norm_forward", "asr_layer_norm_backward", "asr_embedding_forward",
         "asr_embedding_backward", "asr_linear_i8_forward", "asr_linear_i8_backward",
         "asr_linear_i8_forward_saved", "asr_linear_i8_backward_saved"]


@pytest.fixture
def calls(monkeypatch):
    made = []
    for name in NAMES:
        monkeypatch.setattr(_abi, name, lambda *args, name=name: made.append((name, args)))
    for name in [n for n in dir(_abi) if n.endswith("_workspace_bytes")]:
        monkeypatch.setattr(_abi, name, lambda *args: 256)
    monkeypatch.setattr(layers, "_check_floats", lambda *args: None)
    monkeypatch.setattr(int8, "_check_operands", lambda *args: None)
    monkeypatch.setattr(ops, "_on", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(ops, "_stream", lambda device: None)
    return made


def _last(calls, name):
    return [args for n, args in calls if n == name][-1]


def _pass(op, saved):
    """(output, shape of the gradient) of an operator on small CPU tensors."""
    if op == "layer_norm":
        x, w = (torch.randn(*s, requires_grad=True) for s in ((5, 24), (24,)))
        return layer_norm(x * 1.0, w * 1.0, saved=saved)
    if op == "embedding":
        return embedding(torch.arange(6).view(2, 3), torch.randn(9, 24, requires_grad=True))
    x, w = (torch.randn(*s).bfloat16().requires_grad_() for s in ((5, 24), (7, 24)))
    return linear_i8(x * 1.0, w * 1.0, saved=saved)


FORMS = [("layer_norm", "input"), ("layer_norm", "i8"), ("embedding", None),
         ("linear_i8", "input"), ("linear_i8", "i8")]


@pytest.mark.parametrize("op,saved", FORMS)
@pytest.mark.parametrize("kind", ["type", "shape", "device"])
def test_other_tensors_are_refused(calls, op, saved, kind):
    """Each saved tensor in turn comes back as another kind."""
    def change(t):
        if kind == "type":
            return t.to(torch.int16 if t.dtype != torch.int16 else torch.int8)
        return t.to("meta") if kind == "device" else torch.cat([t.flatten(), t.flatten()[:1]])

    saves = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: saves.append(1) or t, lambda t: t):
        _pass(op, saved)
    assert saves
    for k in range(len(saves)):
        seen = []

        def unpack(t):
            seen.append(1)
            return change(t) if len(seen) == k + 1 else t

        with torch.autograd.graph.saved_tensors_hooks(lambda t: t, unpack):
            y = _pass(op, saved)
        before = len(calls)
        with pytest.raises(RuntimeError, match="saved tensor"):
            y.backward(torch.zeros_like(y))
        assert len(calls) == before, k


def _spread(t):
    if t.dim() != 2:
        return t
    wide = t.new_empty((t.shape[0], 2 * t.shape[1] + 16))
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _columns(t):
    return t.t().contiguous().t() if t.dim() == 2 else torch.stack([t, t], -1)[..., 0]


@pytest.mark.parametrize("op,saved", FORMS)
@pytest.mark.parametrize("layout", [_spread, _columns], ids=["spread", "columns"])
def test_other_layouts_are_walked_or_copied(calls, op, saved, layout):
    """The address and stride of each operand belong to one tensor, rows contiguous."""
    got = []

    def unpack(t):
        got.append(layout(t))
        return got[-1]

    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, unpack):
        y = _pass(op, saved)
    y.backward(torch.zeros_like(y))
    name = f"asr_{op}_backward" + ("_saved" if (op, saved) == ("linear_i8", "i8") else "")
    args = _last(calls, name)

    def check(p, ld, t, cols):
        if t.stride(1) == 1:
            assert p == t.data_ptr() and ld == t.stride(0)
        else:
            assert p != t.data_ptr() and ld == cols

    if (op, saved) == ("layer_norm", "input"):
        check(args[2], args[3], got[0], 24)
    if op == "linear_i8":
        if saved == "input":
            check(args[0], args[1], got[0], 24)
            check(args[2], args[3], got[1], 24)
        else:
            check(args[0], args[1], got[0], 32)
            check(args[3], args[4], got[2], 24)
            if layout is _columns:
                assert args[2] != got[1].data_ptr()      # scales side by side
    if op == "embedding" and layout is _columns:
        assert args[0] != got[0].data_ptr()              # ids side by side


def test_codes_keep_their_alignment(calls):
    """Buffers of codes on an address of one byte more: copied to an aligned one."""
    def odd(t):
        if t.dtype not in (torch.uint8, torch.int8):
            return t
        room = t.new_empty(t.numel() + 32)
        skip = 1 + (-room.data_ptr()) % 16
        room[skip:skip + t.numel()] = t.flatten()
        return room[skip:skip + t.numel()].view(t.shape)

    for op, saved, name, at in (("layer_norm", "i8", "asr_layer_norm_backward", 7),
                                ("layer_norm", "input", "asr_layer_norm_backward", 7),
                                ("linear_i8", "i8", "asr_linear_i8_backward_saved", 0)):
        with torch.autograd.graph.saved_tensors_hooks(lambda t: t, odd):
            y = _pass(op, saved)
        y.backward(torch.zeros_like(y))
        assert _last(calls, name)[at] % 16 == 0


def test_linear_asks_for_no_second_room_for_its_codes(monkeypatch, calls):
    """Keeping x's codes, the forward call's workspace is that of one token."""
    asked = []
    monkeypatch.setattr(_abi, "asr_linear_i8_workspace_bytes", lambda *args: asked.append(args) or 256)
    _pass("linear_i8", "i8")
    _pass("linear_i8", "input")
    assert asked == [(1, 7, 24, 0), (5, 7, 24, 0)]


def test_linear_saved_workspace():
    from adamw_optimizer_stochastic_amd import _build
    if not _build.is_built():
        _build.build()
    need = _abi.asr_linear_i8_workspace_bytes(1, 24, 56, 0)
    assert need < _abi.asr_linear_i8_workspace_bytes(400, 24, 56, 0)
    with pytest.raises(_abi.AsrError) as e:
        _abi.asr_linear_i8_forward_saved(0x1000, 56, 0x8000, 56, 0x10000, 24, 0x20000, 64, 0x30000, 400, 24, 56,
                                         0x100000, need - 1, None)
    assert e.value.status == _abi.ASR_EWORKSPACE
