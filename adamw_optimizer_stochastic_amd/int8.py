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
"""

import torch

from . import _abi, ops

__all__ = ["linear_i8"]


class _LinearI8(torch.autograd.Function):
    """x (T, K) and w (N, K), rows contiguous; the checks are linear_i8's."""

    @staticmethod
    def forward(ctx, x, w, grad_rounding, key):
        ctx.save_for_backward(x, w)
        ctx.grad_rounding, ctx.key = grad_rounding, key
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
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, w = ctx.saved_tensors
        (t, k), n, device = x.shape, w.shape[0], x.device
        if dy.stride(1) != 1 or dy.stride(0) < n:
            dy = dy.contiguous()   # an expanded or transposed gradient
        want_x, want_w = ctx.needs_input_grad[:2]
        dx = torch.empty((t, k), dtype=torch.bfloat16, device=device) if want_x else None
        dw = torch.empty((n, k), dtype=torch.bfloat16, device=device) if want_w else None
        need = _abi.asr_linear_i8_workspace_bytes(t, n, k, 1)
        ws = torch.empty(need, dtype=torch.uint8, device=device)
        with ops._on(device):
            _abi.asr_linear_i8_backward(
                x.data_ptr(), ops._row_stride(x, k), w.data_ptr(), ops._row_stride(w, k),
                dy.data_ptr(), ops._row_stride(dy, n), dx.data_ptr() if want_x else None, k,
                dw.data_ptr() if want_w else None, k, t, n, k,
                ops.ROUNDING_CODE[ctx.grad_rounding], *ctx.key, ws.data_ptr(), need,
                ops._stream(device))
        return dx, dw, None, None


def linear_i8(x, w, *, seed=0, step=0, base_index=0, grad_rounding="sr"):
    """y = x w^T in 8-bit integer products, forward and backward.

    x: bfloat16 (..., K); w: bfloat16 (N, K); y: bfloat16 (..., N). The
    gradients are bfloat16. grad_rounding: "sr" (stochastic, under key (seed,
    step), positions from base_index) or "rn", for the gradient's codes; give
    every layer its own base_index (or seed) and every step its own step.
    K, N and the number of tokens are below 2**17 (each is summed over once).

    Forward and backward can be captured into a graph together; as with any
    operator under torch's autograd, no eager graph of the same leaves may be
    alive then (the gradient's accumulation would run on that graph's stream).
    """
    if grad_rounding not in ops.ROUNDING_CODE:
        raise ValueError("grad_rounding must be 'sr' or 'rn'")
    key = (ops._u32("seed", seed), ops._u32("step", step), ops._u64("base_index", base_index))
    for t, name in ((x, "x"), (w, "w")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be bfloat16 (got {t.dtype})")
        if not t.is_cuda:
            raise ValueError(f"{name} must be on a GPU (got {t.device})")
    if x.device != w.device:
        raise ValueError("x and w must be on the same device")
    if x.dim() < 1 or w.dim() != 2 or x.shape[-1] != w.shape[1]:
        raise ValueError(f"x must be (..., K) and w (N, K): got {tuple(x.shape)} and "
                         f"{tuple(w.shape)}")
    n, k = w.shape
    tokens = x.numel() // k if k else x.shape[:-1].numel()
    if max(tokens, n, k) >= 1 << 17:
        raise ValueError("tokens, N and K must be below 2**17")
    flat = x.reshape(tokens, k)
    if flat.numel() and (flat.stride(1) != 1 or flat.stride(0) < k):
        flat = flat.contiguous()
    if w.numel() and (w.stride(1) != 1 or w.stride(0) < k):
        w = w.contiguous()
    if key[2] + tokens * n > 1 << 64:
        raise ValueError("base_index + tokens*N exceeds 2**64")
    y = _LinearI8.apply(flat, w, grad_rounding, key)
    return y.reshape(*x.shape[:-1], n)
