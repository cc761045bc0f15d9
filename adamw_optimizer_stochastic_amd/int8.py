"""A linear layer whose three matrix products run in 8-bit integers.

The layer's weights stay bf16 (the optimizers update them with stochastic
rounding and no f32 master copy); every product quantises its operands on the
way, with one scale for each row of both. Three products, with x (T, K), w
(N, K) and the gradient dy (T, N):

    y  = x  w^T    sums over K: scales for each token of x and channel of w
    dx = dy w      sums over N: scales for each token of dy and input of w
    dw = dy^T x    sums over T: scales for each output of dy and input of x

x and w are rounded to nearest. dy is rounded stochastically (by default):
its codes are then unbiased, so the quantisation of dy adds no bias to dx or
dw. Element (t, n) of dy uses stream position base_index + t*N + n under key
(seed, step), in both products.

With saved="i8" the layer keeps x's codes of the first product, one byte an
element, instead of x. The third product takes them as they are: x is about s[t]
X[t, k], so the token's scale goes into dy before dy's column codes are taken,

    dw = (s dy)^T X   scales for each output of s dy, X's codes turned round

and x is rounded once, not a second time along its columns.
"""

import torch

from . import _abi, ops

__all__ = ["linear_i8"]


def _check_operands(x, w):
    for t, name in ((x, "x"), (w, "w")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be bfloat16 (got {t.dtype})")
        if not t.is_cuda:
            raise ValueError(f"{name} must be on a GPU (got {t.device})")
    if x.device != w.device:
        raise ValueError("x and w must be on the same device")


def _rows(t):
    """(tensor, row stride): the matrix t, or a copy of it if its rows are not contiguous
    or overlap."""
    if t.is_contiguous():
        return t, max(t.shape[1], 1)
    if t.numel() and (t.stride(1) != 1 or t.stride(0) < t.shape[1]):
        t = t.contiguous()
    return t, ops._row_stride(t, t.shape[1])


def _kept_rows(t, device, dtype, rows, cols):
    """_rows of a matrix that a pass kept (ops._kept), in any layout."""
    ops._kept(t, device, dtype, rows * cols)
    if t.shape != (rows, cols):
        raise RuntimeError(f"a saved tensor came back as {tuple(t.shape)}, not as {(rows, cols)}")
    return _rows(t)


class _LinearI8(torch.autograd.Function):
    """x (T, K) and w (N, K), rows contiguous; the checks are linear_i8's."""

    @staticmethod
    def forward(ctx, x, w, grad_rounding, key):
        ctx.save_for_backward(x, w)
        ctx.width, ctx.grad_rounding, ctx.key = x.shape[1], grad_rounding, key
        (t, k), n, device = x.shape, w.shape[0], x.device
        y = torch.empty((t, n), dtype=torch.bfloat16, device=device)
        need = _abi.asr_linear_i8_workspace_bytes(t, n, k, 0)
        ws = torch.empty(need, dtype=torch.uint8, device=device)
        with ops._on(device):
            _abi.asr_linear_i8_forward(x.data_ptr(), ops._row_stride(x, k), w.data_ptr(),
                                       ops._row_stride(w, k), y.data_ptr(), n, t, n, k,
                                       ws.data_ptr(), need, ops._stream(device))
        return y

    @staticmethod
    @ops._once
    def backward(ctx, dy):
        x, w = ctx.saved_tensors
        (t, n), k, device = dy.shape, ctx.width, dy.device
        dy, ld_dy = _rows(dy)   # (an expanded or transposed gradient)
        x, ld_x = _kept_rows(x, device, torch.bfloat16, t, k)
        w, ld_w = _kept_rows(w, device, torch.bfloat16, n, k)
        want_x, want_w = ctx.needs_input_grad[:2]
        dx = dy.new_empty((t, k)) if want_x else None
        dw = dy.new_empty((n, k)) if want_w else None
        need = _abi.asr_linear_i8_workspace_bytes(t, n, k, 1)
        ws = torch.empty(need, dtype=torch.uint8, device=device)
        with ops._on(device):
            _abi.asr_linear_i8_backward(
                x.data_ptr(), ld_x, w.data_ptr(), ld_w, dy.data_ptr(), ld_dy,
                dx.data_ptr() if want_x else None, k, dw.data_ptr() if want_w else None, k, t, n, k,
                ops.ROUNDING_CODE[ctx.grad_rounding], *ctx.key, ws.data_ptr(), need,
                ops._stream(device))
        return dx, dw, None, None


class _LinearI8Saved(torch.autograd.Function):
    """The same, keeping x's codes instead of x."""

    @staticmethod
    def forward(ctx, x, w, grad_rounding, key):
        (t, k), n, device = x.shape, w.shape[0], x.device
        y = torch.empty((t, n), dtype=torch.bfloat16, device=device)
        q = torch.empty((t, max(ops._padded16(k), 16)), dtype=torch.int8, device=device)
        scale = torch.empty(t, dtype=torch.float32, device=device)
        ctx.save_for_backward(q, scale, w)
        ctx.width, ctx.grad_rounding, ctx.key = k, grad_rounding, key
        need = _abi.asr_linear_i8_workspace_bytes(1, n, k, 0)   # (x's codes are in q)
        ws = torch.empty(need, dtype=torch.uint8, device=device)
        with ops._on(device):
            _abi.asr_linear_i8_forward_saved(
                x.data_ptr(), ops._row_stride(x, k), w.data_ptr(), ops._row_stride(w, k),
                y.data_ptr(), n, q.data_ptr(), q.shape[1], scale.data_ptr(), t, n, k,
                ws.data_ptr(), need, ops._stream(device))
        return y

    @staticmethod
    @ops._once
    def backward(ctx, dy):
        q, scale, w = ctx.saved_tensors
        (t, n), k, device = dy.shape, ctx.width, dy.device
        dy, ld_dy = _rows(dy)   # (an expanded or transposed gradient)
        w, ld_w = _kept_rows(w, device, torch.bfloat16, n, k)
        scale = ops._kept(scale, device, torch.float32, t).contiguous()
        width = max(ops._padded16(k), 16)
        q, ld_q = _kept_rows(q, device, torch.int8, t, width)
        if q.data_ptr() % 16 or ld_q % 16:
            q, ld_q = q.clone(memory_format=torch.contiguous_format), width
        want_x, want_w = ctx.needs_input_grad[:2]
        dx = dy.new_empty((t, k)) if want_x else None
        dw = dy.new_empty((n, k)) if want_w else None
        need = _abi.asr_linear_i8_workspace_bytes(t, n, k, 1)
        ws = torch.empty(need, dtype=torch.uint8, device=device)
        with ops._on(device):
            _abi.asr_linear_i8_backward_saved(
                q.data_ptr(), ld_q, scale.data_ptr(), w.data_ptr(), ld_w, dy.data_ptr(), ld_dy,
                dx.data_ptr() if want_x else None, k, dw.data_ptr() if want_w else None, k, t, n, k,
                ops.ROUNDING_CODE[ctx.grad_rounding], *ctx.key, ws.data_ptr(), need,
                ops._stream(device))
        return dx, dw, None, None


def linear_i8(x, w, *, seed=0, step=0, base_index=0, grad_rounding="sr", saved="input"):
    """y = x w^T in 8-bit integer products, forward and backward.

    x: bfloat16 (..., K); w: bfloat16 (N, K); y: bfloat16 (..., N). The
    gradients are bfloat16. grad_rounding: "sr" (stochastic, under key (seed,
    step), positions from base_index) or "rn", for the gradient's codes; give
    every layer its own base_index (or seed) and every step its own step.
    K, N and the number of tokens are below 2**17 (each is summed over once).
    saved: "input" keeps x for w's gradient, "i8" the codes of the forward
    product (half the bytes; y and dx are the same, and a token with an Inf or
    NaN in x makes all of w's gradient NaN).

    Forward and backward can be captured into a graph together; as with any
    operator under torch's autograd, no eager graph of the same leaves may be
    alive then (the gradient's accumulation would run on that graph's stream).
    """
    if grad_rounding not in ops.ROUNDING_CODE:
        raise ValueError("grad_rounding must be 'sr' or 'rn'")
    if saved not in ("input", "i8"):
        raise ValueError("saved must be 'input' or 'i8'")
    key = (ops._u32("seed", seed), ops._u32("step", step), ops._u64("base_index", base_index))
    _check_operands(x, w)
    if x.dim() < 1 or w.dim() != 2 or x.shape[-1] != w.shape[1]:
        raise ValueError(f"x must be (..., K) and w (N, K): got {tuple(x.shape)} and "
                         f"{tuple(w.shape)}")
    n, k = w.shape
    tokens = x.numel() // k if k else x.shape[:-1].numel()
    if max(tokens, n, k) >= 1 << 17:
        raise ValueError("tokens, N and K must be below 2**17")
    flat = x if x.dim() == 2 else x.reshape(tokens, k)
    flat, w = _rows(flat)[0], _rows(w)[0]
    if key[2] + tokens * n > 1 << 64:
        raise ValueError("base_index + tokens*N exceeds 2**64")
    layer = _LinearI8Saved if saved == "i8" and n > 0 and k > 0 else _LinearI8
    y = layer.apply(flat, w, grad_rounding, key)
    return y if x.dim() == 2 else y.reshape(*x.shape[:-1], n)
