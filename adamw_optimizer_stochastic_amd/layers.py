"""The layers between a model's products: embedding, layer norm, gated SiLU.

Each is a function with its gradients (torch's autograd) on the library's
kernels, for float32 and bfloat16. ``layer_norm`` and ``silu_mul`` can keep what
their backward pass needs as 8-bit codes with one scale for every 128 columns
(``ops.pack_i8``'s, 1.03 bytes an element) instead of their inputs; the
gradients are then the formulas' at the values the codes stand for. Forward
and backward can be captured into a graph together; as with any operator under
torch's autograd, no eager graph of the same leaves may be alive then. Forward-mode
derivatives, second derivatives and torch.func's transforms raise.
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


def _matrix(t, cols):
    """(tensor, rows, row stride) of t as a matrix of rows of `cols` contiguous
    elements: t itself where it is contiguous (no view is made: each costs a
    microsecond, and a node of autograd's graph), else a view or a copy."""
    if t.is_contiguous():
        return t, (t.numel() // cols if cols else t.shape[:-1].numel()), max(cols, 1)
    flat = t.reshape(t.shape[:-1].numel(), cols)
    if flat.numel() and ((cols > 1 and flat.stride(1) != 1) or
                         (flat.shape[0] > 1 and flat.stride(0) < cols)):
        flat = flat.contiguous()
    return flat, flat.shape[0], ops._row_stride(flat, cols)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _kept_matrix(t, like, rows, cols):
    """(tensor, row stride) of a matrix that a pass kept (ops._kept), in any layout."""
    ops._kept(t, like.device, like.dtype, rows * cols)
    if t.shape[-1:] != (cols,):
        raise RuntimeError(f"a saved tensor came back as {tuple(t.shape)}, not as (..., {cols})")
    if t.is_contiguous():
        return t, max(cols, 1)
    flat, _, ld = _matrix(t, cols)
    return flat, ld


class _Codes:
    """The buffers a pass keeps for its backward pass, in one allocation: `head`
    bytes, then scales and codes of `count` matrices of rows x cols."""

    def __init__(self, rows, cols, count, head=0):
        self.ld = max(ops._padded16(cols), 16)
        self.scale = head
        self.step = ops._padded16(rows * ((cols + ops.PACK_COLUMNS - 1) // ops.PACK_COLUMNS) * 4)
        self.codes = head + count * self.step
        self.size = rows * self.ld
        self.bytes = self.codes + count * self.size

    def at(self, base, k):
        """(codes, scales) of matrix k in the buffer at address base."""
        return base + self.codes + k * self.size, base + self.scale + k * self.step


# ---------------------------------------------------------- layer norm
def _norm_forward(x, weight, bias, eps, keep, codes):
    """(y, what the backward pass needs, x as a matrix or None)."""
    cols, device = x.shape[-1], x.device
    flat, rows, ld = _matrix(x, cols)
    y = torch.empty_like(x) if flat is x else torch.empty(x.shape, dtype=x.dtype, device=device)
    buffer = stat = q = scale = None
    ldq = 0
    if codes:
        layout = _Codes(rows, cols, 1, 16 * rows)
        buffer = torch.empty(layout.bytes, dtype=torch.uint8, device=device)
        stat = buffer.data_ptr()
        (q, scale), ldq = layout.at(stat, 0), layout.ld
    elif keep:
        buffer = torch.empty(16 * rows, dtype=torch.uint8, device=device)
        stat = buffer.data_ptr()
    param = weight if weight is not None else bias
    with ops._on(device):
        _abi.asr_layer_norm_forward(
            flat.data_ptr(), ops._DTYPE_CODE[x.dtype], ld, rows, cols, _ptr(weight), _ptr(bias),
            ops._DTYPE_CODE[x.dtype if param is None else param.dtype], eps, y.data_ptr(), stat,
            q, ldq, scale, ops._stream(device))
    return y, buffer, None if codes else flat


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, saved):
        y, buffer, flat = _norm_forward(x, weight, bias, eps, True, saved == "i8")
        ctx.save_for_backward(flat, weight, buffer)
        param = weight if weight is not None else bias
        ctx.param_dtype = None if param is None else param.dtype
        return y

    @staticmethod
    @ops._once
    def backward(ctx, dy):
        x, weight, buffer = ctx.saved_tensors
        cols, device, dtype = dy.shape[-1], dy.device, dy.dtype
        flat, rows, ld = _matrix(dy, cols)
        want_x, want_w, want_b = ctx.needs_input_grad[:3]
        pdt = ctx.param_dtype or dtype
        if weight is not None:
            weight = ops._kept(weight, device, pdt, cols).contiguous()
        dx = dy.new_empty(dy.shape) if want_x else None
        dw = torch.empty_like(weight) if want_w else None
        db = torch.empty(cols, dtype=pdt, device=device) if want_b else None
        x_ptr, ldx, q, scale, ldq = None, 0, None, None, 0
        if x is None:
            layout = _Codes(rows, cols, 1, 16 * rows)
            buffer = ops._kept_buffer(buffer, device, layout.bytes)
            (q, scale), ldq = layout.at(buffer.data_ptr(), 0), layout.ld
        else:
            buffer = ops._kept_buffer(buffer, device, 16 * rows)
            x, ldx = _kept_matrix(x, dy, rows, cols)
            x_ptr = x.data_ptr()
        stat = buffer.data_ptr()
        need, ws = 0, None
        if want_w or want_b:
            need = _abi.asr_layer_norm_backward_workspace_bytes(rows, cols)
            ws = torch.empty(need, dtype=torch.uint8, device=device)
        with ops._on(device):
            _abi.asr_layer_norm_backward(
                flat.data_ptr(), ld, x_ptr, ldx, q, ldq, scale, stat, ops._DTYPE_CODE[dtype],
                rows, cols, _ptr(weight), ops._DTYPE_CODE[pdt], _ptr(dx), _ptr(dw), _ptr(db),
                _ptr(ws), need, ops._stream(device))
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
    with an Inf or NaN gives NaN; x - mean is formed in binary32 and has to fit
    there, as has 1 / sqrt(var + eps). Up to 2**24 columns, fewer than 2**24 rows.
    """
    if saved not in ("input", "i8"):
        raise ValueError("saved must be 'input' or 'i8'")
    eps = float(eps)
    if not (eps >= 0.0 and math.isfinite(eps)):
        raise ValueError("eps must be finite and >= 0")
    _check_floats(x, "x")
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    cols, device = x.shape[-1], x.device
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _check_floats(t, name, device)
            if t.dim() != 1 or t.shape[0] != cols:
                raise ValueError(f"{name} must have shape ({cols},)")
    if weight is not None:
        if bias is not None and weight.dtype != bias.dtype:
            raise TypeError("weight and bias must have the same type")
        if not weight.is_contiguous():
            weight = weight.contiguous()
    if bias is not None and not bias.is_contiguous():
        bias = bias.contiguous()
    if cols > 1 << 24 or (x.numel() // cols if cols else x.shape[:-1].numel()) >= 1 << 24:
        raise ValueError("fewer than 2**24 rows and at most 2**24 columns")
    if ops._dual_level() or torch.is_grad_enabled() and (
            x.requires_grad or (weight is not None and weight.requires_grad)
            or (bias is not None and bias.requires_grad)):
        return _LayerNorm.apply(x, weight, bias, eps, saved)
    return _norm_forward(x, weight, bias, eps, False, False)[0]


# ----------------------------------------------------------- gated SiLU
def _silu_forward(gate, up, codes):
    """(y, codes' buffer or None, gate and up as matrices)."""
    width, device, dtype = gate.shape[-1], gate.device, gate.dtype
    flat, rows, ld = _matrix(gate, width)
    if up is None:   # the halves of gate's columns
        cols, u, ld_u = width // 2, None, ld
        g_ptr = flat.data_ptr()
        u_ptr = g_ptr + cols * flat.element_size()
    else:
        cols = width
        u, _, ld_u = _matrix(up, cols)
        g_ptr, u_ptr = flat.data_ptr(), u.data_ptr()
    y = torch.empty((*gate.shape[:-1], cols), dtype=dtype, device=device)
    buffer, ldq = None, 0
    pointers = (None,) * 4
    if codes:
        layout = _Codes(rows, cols, 2)
        buffer = torch.empty(layout.bytes, dtype=torch.uint8, device=device)
        base, ldq = buffer.data_ptr(), layout.ld
        pointers = (*layout.at(base, 0), *layout.at(base, 1))
    with ops._on(device):
        _abi.asr_silu_mul_forward(g_ptr, ld, u_ptr, ld_u, ops._DTYPE_CODE[dtype], rows, cols,
                                  y.data_ptr(), max(cols, 1), *pointers, ldq,
                                  ops._stream(device))
    return y, buffer, flat, u


class _SiluMul(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate, up, saved):
        codes = saved == "i8"
        y, buffer, g, u = _silu_forward(gate, up, codes)
        ctx.joint = up is None
        ctx.save_for_backward(None if codes else g, None if codes else u, buffer)
        return y

    @staticmethod
    @ops._once
    def backward(ctx, dy):
        gate, up, buffer = ctx.saved_tensors
        cols, device, dtype = dy.shape[-1], dy.device, dy.dtype
        flat, rows, ld = _matrix(dy, cols)
        half = cols * flat.element_size()
        if ctx.joint:
            dgate = torch.empty((*dy.shape[:-1], 2 * cols), dtype=dtype, device=device)
            dup, ld_out = None, max(2 * cols, 1)
            out_g = dgate.data_ptr()
            out_u = out_g + half
        else:
            dgate, dup = (torch.empty(dy.shape, dtype=dtype, device=device) for _ in range(2))
            out_g, out_u, ld_out = dgate.data_ptr(), dup.data_ptr(), max(cols, 1)
        pointers, ldq, g, ld_g, u, ld_u = (None,) * 4, 0, None, 0, None, 0
        if buffer is not None:
            layout = _Codes(rows, cols, 2)
            buffer = ops._kept_buffer(buffer, device, layout.bytes)
            base, ldq = buffer.data_ptr(), layout.ld
            pointers = (*layout.at(base, 0), *layout.at(base, 1))
        else:
            gate, ld_g = _kept_matrix(gate, dy, rows, 2 * cols if ctx.joint else cols)
            g = gate.data_ptr()
            if ctx.joint:
                u, ld_u = g + half, ld_g
            else:
                up, ld_u = _kept_matrix(up, dy, rows, cols)
                u = up.data_ptr()
        with ops._on(device):
            _abi.asr_silu_mul_backward(flat.data_ptr(), ld, g, ld_g, u, ld_u, *pointers, ldq,
                                       ops._DTYPE_CODE[dtype], rows, cols, out_g, ld_out, out_u,
                                       ld_out, ops._stream(device))
        return dgate, dup, None


def silu_mul(gate, up=None, *, saved="inputs"):
    """silu(gate) * up, the gated activation of an MLP; silu(g) = g / (1 + exp(-g)).

    gate, up: float32 or bfloat16 of one type and shape (..., C). Without ``up``,
    gate is (..., 2C), a product with both weights at once: its first C columns
    are the gate, the others up, and its gradient is one tensor too. Rows may
    have any stride (those that are not contiguous are copied).

    saved: "inputs" keeps gate and up for the backward pass; "i8" their 8-bit
    codes (``ops.pack_i8``'s, to nearest), and takes the gradients from what
    these stand for. Both gradients are computed together. Where the sigmoid is
    below 2**-126 (a gate under -87) it may be taken as 0.
    """
    if saved not in ("inputs", "i8"):
        raise ValueError("saved must be 'inputs' or 'i8'")
    _check_floats(gate, "gate")
    if gate.dim() < 1:
        raise ValueError("gate must have at least one dimension")
    if up is None:
        if gate.shape[-1] % 2:
            raise ValueError("without up, gate's last dimension must be even")
    else:
        _check_floats(up, "up", gate.device, gate.dtype)
        if up.shape != gate.shape:
            raise ValueError("gate and up must have the same shape")
    if ops._dual_level() or torch.is_grad_enabled() and (
            gate.requires_grad or (up is not None and up.requires_grad)):
        return _SiluMul.apply(gate, up, saved)
    return _silu_forward(gate, up, False)[0]


# ------------------------------------------------------------ embedding
def _lookup(ids, weight, scale):
    (vocab, dim), device = weight.shape, weight.device
    y = torch.empty((*ids.shape, dim), dtype=weight.dtype, device=device)
    table, _, ld = _matrix(weight, dim)
    with ops._on(device):
        _abi.asr_embedding_forward(ids.data_ptr(), int(ids.dtype == torch.int64), ids.numel(),
                                   table.data_ptr(), ops._DTYPE_CODE[weight.dtype], ld, vocab, dim,
                                   scale, y.data_ptr(), ops._stream(device))
    return y


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, ids, scale, padding):
        ctx.save_for_backward(ids)
        ctx.args = weight.shape, scale, padding, ids.dtype
        return _lookup(ids, weight, scale)

    @staticmethod
    @ops._once
    def backward(ctx, dy):
        ids, = ctx.saved_tensors
        (vocab, dim), scale, padding, id_type = ctx.args
        flat, n, ld = _matrix(dy, dim)
        device = dy.device
        ids = ops._kept(ids, device, id_type, n).contiguous()
        dw = dy.new_empty((vocab, dim))
        need = _abi.asr_embedding_backward_workspace_bytes(n, vocab, dim)
        ws = torch.empty(need, dtype=torch.uint8, device=device) if need else None
        with ops._on(device):
            _abi.asr_embedding_backward(
                ids.data_ptr(), int(id_type == torch.int64), n, flat.data_ptr(), ld,
                ops._DTYPE_CODE[dy.dtype], vocab, dim, scale, padding, dw.data_ptr(),
                _ptr(ws), need, ops._stream(device))
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
    if not ids.is_contiguous():
        ids = ids.contiguous()
    if ops._dual_level() or torch.is_grad_enabled() and weight.requires_grad:
        return _Embedding.apply(weight, ids, scale, padding)
    return _lookup(ids, weight, scale)
