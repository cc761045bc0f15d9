"""The layers between a model's products: embedding, layer norm, gated SiLU.

Each is a function with its gradients (torch's autograd) on the library's
kernels, for float32 and bfloat16. ``layer_norm`` and ``silu_mul`` can keep what
their backward pass needs as 8-bit codes with one scale for every 128 columns
(``ops.pack_i8``'s, 1.03 bytes an element) instead of their inputs; the
gradients are then the formulas' at the values the codes stand for. Forward
and backward can be captured into a graph together; as with any operator under
torch's autograd, no eager graph of the same leaves may be alive then.
"""

import math
import operator

import torch

from . import _abi, ops

__all__ = ["embedding", "layer_norm", "silu_mul"]

_FLOATS = (torch.float32, torch.bfloat16)


def _check_floats(t, name, device=None, dtype=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU (got {t.device})")
    if t.dtype not in _FLOATS:
        raise TypeError(f"{name} must be float32 or bfloat16 (got {t.dtype})")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device} (got {t.device})")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")


def _rows(t, cols):
    """t as a matrix of rows of `cols` contiguous elements (a copy where t's
    strides do not allow it)."""
    if t.is_contiguous():
        return t.view(-1, cols) if cols else t.reshape(t.shape[:-1].numel(), 0)
    flat = t.reshape(t.shape[:-1].numel(), cols)
    if flat.numel() and ((cols > 1 and flat.stride(1) != 1) or
                         (flat.shape[0] > 1 and flat.stride(0) < cols)):
        flat = flat.contiguous()
    return flat


def _wants_grad(*tensors):
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


def _ptr(t):
    return None if t is None else t.data_ptr()


# ---------------------------------------------------------- layer norm
def _norm_forward(x, weight, bias, eps, keep, codes):
    """(y, stat, q, scale) of a matrix; stat with `keep`, the codes with `codes`."""
    (rows, cols), device = x.shape, x.device
    y = torch.empty((rows, cols), dtype=x.dtype, device=device)
    stat = torch.empty((rows, 4), dtype=torch.float32, device=device) if keep else None
    q, scale = ops._code_buffers(rows, cols, device) if codes else (None, None)
    param = weight if weight is not None else bias
    with ops._on(device):
        _abi.asr_layer_norm_forward(
            x.data_ptr(), ops._DTYPE_CODE[x.dtype], ops._row_stride(x, cols), rows, cols,
            _ptr(weight), _ptr(bias), ops._DTYPE_CODE[x.dtype if param is None else param.dtype],
            eps, y.data_ptr(), _ptr(stat), _ptr(q), q.shape[1] if codes else 0, _ptr(scale),
            ops._stream(device))
    return y, stat, q, scale


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, saved):
        codes = saved == "i8"
        y, stat, q, scale = _norm_forward(x, weight, bias, eps, True, codes)
        ctx.save_for_backward(None if codes else x, weight, stat, q, scale)
        ctx.bias_dtype = None if bias is None else bias.dtype
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, weight, stat, q, scale = ctx.saved_tensors
        rows, cols = dy.shape
        dy, device = _rows(dy, cols), dy.device
        want_x, want_w, want_b = ctx.needs_input_grad[:3]
        pdt = dy.dtype
        if weight is not None or ctx.bias_dtype is not None:
            pdt = weight.dtype if weight is not None else ctx.bias_dtype
        dx = torch.empty((rows, cols), dtype=dy.dtype, device=device) if want_x else None
        dw = torch.empty(cols, dtype=pdt, device=device) if want_w else None
        db = torch.empty(cols, dtype=pdt, device=device) if want_b else None
        need, ws = 0, None
        if want_w or want_b:
            need = _abi.asr_layer_norm_backward_workspace_bytes(rows, cols)
            ws = torch.empty(need, dtype=torch.uint8, device=device)
        with ops._on(device):
            _abi.asr_layer_norm_backward(
                dy.data_ptr(), ops._row_stride(dy, cols), _ptr(x),
                ops._row_stride(x, cols) if x is not None else 0, _ptr(q),
                q.shape[1] if q is not None else 0, _ptr(scale), stat.data_ptr(),
                ops._DTYPE_CODE[dy.dtype], rows, cols, _ptr(weight), ops._DTYPE_CODE[pdt],
                _ptr(dx), _ptr(dw), _ptr(db), _ptr(ws), need, ops._stream(device))
        return dx, dw, db, None, None


def layer_norm(x, weight=None, bias=None, eps=1e-5, *, saved="input"):
    """Layer norm over the last dimension: (x - mean) / sqrt(var + eps) * weight + bias.

    x: float32 or bfloat16 (..., C), any strides (rows that are not contiguous
    are copied); weight, bias: None or (C,), float32 or bfloat16, both of one
    type. The result has x's type, the gradients those of their inputs. mean
    and var are formed in 64 bits; the sums over rows for weight and bias take an order that
    depends on the sizes only, so equal calls give equal bits.

    saved: "input" keeps x for the backward pass; "i8" keeps the 8-bit codes of
    the normalised rows (``ops.pack_i8``'s of their 64-bit values), a half or a
    quarter of x's bytes, and takes the gradients from what they stand for. A row
    with an Inf or NaN gives NaN. Up to 2**24 columns, fewer than 2**24 rows.
    """
    if saved not in ("input", "i8"):
        raise ValueError("saved must be 'input' or 'i8'")
    eps = float(eps)
    if not (eps >= 0.0 and math.isfinite(eps)):
        raise ValueError("eps must be finite and >= 0")
    _check_floats(x, "x")
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    shape, cols, device = x.shape, x.shape[-1], x.device
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _check_floats(t, name, device)
            if t.dim() != 1 or t.shape[0] != cols:
                raise ValueError(f"{name} must have shape ({cols},)")
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError("weight and bias must have the same type")
    if weight is not None and not weight.is_contiguous():
        weight = weight.contiguous()
    if bias is not None and not bias.is_contiguous():
        bias = bias.contiguous()
    flat = _rows(x, cols)
    if flat.shape[0] >= 1 << 24 or cols > 1 << 24:
        raise ValueError("fewer than 2**24 rows and at most 2**24 columns")
    if _wants_grad(x, weight, bias):
        return _LayerNorm.apply(flat, weight, bias, eps, saved).reshape(shape)
    return _norm_forward(flat, weight, bias, eps, False, False)[0].view(shape)


# ----------------------------------------------------------- gated SiLU
def _halves(gate, up):
    """(gate, up, their row strides, cols); up None: the halves of gate's columns."""
    if up is not None:
        cols = gate.shape[1]
        return (gate.data_ptr(), up.data_ptr(), ops._row_stride(gate, cols),
                ops._row_stride(up, cols), cols)
    cols = gate.shape[1] // 2
    ld = ops._row_stride(gate, 2 * cols)
    return gate.data_ptr(), gate.data_ptr() + cols * gate.element_size(), ld, ld, cols


def _silu_forward(gate, up, codes):
    g, u, ld_g, ld_u, cols = _halves(gate, up)
    rows, device = gate.shape[0], gate.device
    y = torch.empty((rows, cols), dtype=gate.dtype, device=device)
    (qg, sg), (qu, su) = ((ops._code_buffers(rows, cols, device) for _ in range(2)) if codes
                          else ((None, None),) * 2)
    with ops._on(device):
        _abi.asr_silu_mul_forward(g, ld_g, u, ld_u, ops._DTYPE_CODE[gate.dtype], rows, cols,
                                  y.data_ptr(), max(cols, 1), _ptr(qg), _ptr(sg), _ptr(qu),
                                  _ptr(su), qg.shape[1] if codes else 0, ops._stream(device))
    return y, qg, sg, qu, su


class _SiluMul(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate, up, saved):
        codes = saved == "i8"
        y, *packed = _silu_forward(gate, up, codes)
        ctx.joint = up is None
        ctx.save_for_backward(*((None, None) if codes else (gate, up)), *packed)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        gate, up, qg, sg, qu, su = ctx.saved_tensors
        rows, cols = dy.shape
        dy, device = _rows(dy, cols), dy.device
        if ctx.joint:
            dgate = torch.empty((rows, 2 * cols), dtype=dy.dtype, device=device)
            dup = None
        else:
            dgate, dup = (torch.empty((rows, cols), dtype=dy.dtype, device=device)
                          for _ in range(2))
        out_g, out_u, ld_dg, ld_du, _ = _halves(dgate, dup)
        g, u, ld_g, ld_u = _halves(gate, up)[:4] if gate is not None else (None, None, 0, 0)
        with ops._on(device):
            _abi.asr_silu_mul_backward(
                dy.data_ptr(), ops._row_stride(dy, cols), g, ld_g, u, ld_u, _ptr(qg), _ptr(sg),
                _ptr(qu), _ptr(su), qg.shape[1] if qg is not None else 0,
                ops._DTYPE_CODE[dy.dtype], rows, cols, out_g, ld_dg, out_u, ld_du,
                ops._stream(device))
        return dgate, dup, None


def silu_mul(gate, up=None, *, saved="inputs"):
    """silu(gate) * up, the gated activation of an MLP; silu(g) = g / (1 + exp(-g)).

    gate, up: float32 or bfloat16 of one type and shape (..., C). Without ``up``,
    gate is (..., 2C), a product with both weights at once: its first C columns
    are the gate, the others up, and its gradient is one tensor too. Rows may
    have any stride (those that are not contiguous are copied).

    saved: "inputs" keeps gate and up for the backward pass; "i8" their 8-bit
    codes (``ops.pack_i8``'s, to nearest), and takes the gradients from what
    these stand for.
    """
    if saved not in ("inputs", "i8"):
        raise ValueError("saved must be 'inputs' or 'i8'")
    _check_floats(gate, "gate")
    if gate.dim() < 1:
        raise ValueError("gate must have at least one dimension")
    width = gate.shape[-1]
    if up is None:
        if width % 2:
            raise ValueError("without up, gate's last dimension must be even")
        cols = width // 2
    else:
        cols = width
        _check_floats(up, "up", gate.device, gate.dtype)
        if up.shape != gate.shape:
            raise ValueError("gate and up must have the same shape")
    shape = (*gate.shape[:-1], cols)
    g, u = _rows(gate, width), None if up is None else _rows(up, width)
    if _wants_grad(gate, up):
        return _SiluMul.apply(g, u, saved).reshape(shape)
    return _silu_forward(g, u, False)[0].view(shape)


# ------------------------------------------------------------ embedding
def _lookup(ids, weight, scale):
    (vocab, dim), device = weight.shape, weight.device
    y = torch.empty((ids.numel(), dim), dtype=weight.dtype, device=device)
    with ops._on(device):
        _abi.asr_embedding_forward(ids.data_ptr(), int(ids.dtype == torch.int64), ids.numel(),
                                   weight.data_ptr(), ops._DTYPE_CODE[weight.dtype],
                                   ops._row_stride(weight, dim), vocab, dim, scale, y.data_ptr(),
                                   ops._stream(device))
    return y


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, ids, scale, padding):
        ctx.save_for_backward(ids)
        ctx.args = weight.shape, scale, padding
        return _lookup(ids, weight, scale)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        ids, = ctx.saved_tensors
        (vocab, dim), scale, padding = ctx.args
        dy, device, n = _rows(dy, dim), dy.device, ids.numel()
        dw = torch.empty((vocab, dim), dtype=dy.dtype, device=device)
        need = _abi.asr_embedding_backward_workspace_bytes(n, vocab, dim)
        ws = torch.empty(need, dtype=torch.uint8, device=device)
        with ops._on(device):
            _abi.asr_embedding_backward(
                ids.data_ptr(), int(ids.dtype == torch.int64), n, dy.data_ptr(),
                ops._row_stride(dy, dim), ops._DTYPE_CODE[dy.dtype], vocab, dim, scale, padding,
                dw.data_ptr(), ws.data_ptr(), need, ops._stream(device))
        return dw, None, None, None


def embedding(ids, weight, *, scale=1.0, padding_idx=None):
    """scale * weight[ids]: rows of a table, float32 or bfloat16, (V, D).

    ids: int64 or int32, any shape; the result is (*ids.shape, D) of weight's
    type, scaled in float32 and rounded once. The gradient of weight is dense:
    for each row scale times the sum of its tokens' gradients, in float32 and
    rounded once, its additions in an order that ids fixes, so equal calls give
    equal bits. padding_idx: an id (negative: from the end) that gets no
    gradient. An id outside [0, V) gives a row of NaN and no gradient (the check
    would have to wait for the GPU).
    """
    _check_floats(weight, "weight")
    if weight.dim() != 2:
        raise ValueError("weight must be (V, D)")
    if not isinstance(ids, torch.Tensor):
        raise TypeError("ids must be a torch.Tensor")
    if ids.dtype not in (torch.int64, torch.int32):
        raise TypeError(f"ids must be int64 or int32 (got {ids.dtype})")
    if ids.device != weight.device:
        raise ValueError(f"ids must be on {weight.device} (got {ids.device})")
    scale = float(scale)
    if not abs(scale) <= 3.4028234663852886e38:
        raise ValueError("scale must be finite in binary32")
    vocab, dim = weight.shape
    padding = -1
    if padding_idx is not None:
        padding = operator.index(padding_idx)
        if not -vocab <= padding < vocab:
            raise ValueError("padding_idx must be an id of the table")
        padding %= vocab
    if not weight.is_contiguous():
        weight = _rows(weight, dim)
    flat = ids.reshape(-1)
    if not flat.is_contiguous():
        flat = flat.contiguous()
    if _wants_grad(weight):
        y = _Embedding.apply(weight, flat, scale, padding)
    else:
        y = _lookup(flat, weight, scale)
    return y.view(*ids.shape, dim)
