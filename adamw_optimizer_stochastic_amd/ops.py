"""Tensor-level entry points over the C ABI (torch supplies memory and streams).

Each function checks devices, dtypes, sizes and contiguity, then calls the
C entry point of the same name (without the ``asr_`` prefix) on the current
HIP stream of the tensors' device. All arithmetic runs in the library's
kernels; there is no CPU path.
"""

import contextlib
import operator

import numpy as np
import torch

from . import _abi
from ._abi import ASR_F32, ASR_BF16, ASR_ROUND_SR, ASR_ROUND_RN, AsrError  # noqa: F401

_DTYPE_CODE = {torch.float32: ASR_F32, torch.bfloat16: ASR_BF16}
ROUNDING_CODE = {"sr": ASR_ROUND_SR, "rn": ASR_ROUND_RN}


def _require_gpu(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU (got {t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# torch's own short way to the current stream's handle, where it has one
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device):
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


# The kernels write through addresses, which autograd does not see: without this
# a backward pass would use the new values of what it saved. Called with every
# list of the caller's tensors that a call has written (42 us for 873 tensors).
_written = torch.autograd.graph.increment_version


_HERE = contextlib.nullcontext()


def _on(device):
    """A context in which `device` is the current one (no more than a
    comparison where it is already)."""
    return _HERE if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _uint(name, x, bits):
    """x as a Python int in [0, 2**bits) (the C argument's range), else
    ValueError: ctypes would otherwise wrap it silently."""
    try:
        v = operator.index(x)
    except TypeError:
        raise TypeError(f"{name} must be an integer (got {type(x).__name__})") from None
    if not 0 <= v < (1 << bits):
        raise ValueError(f"{name} must be in [0, 2**{bits})")
    return v


def _u32(name, x):
    return _uint(name, x, 32)


def _u64(name, x):
    return _uint(name, x, 64)


def check_disjoint(spans):
    """Raise ValueError if any two of the byte ranges overlap. spans: an
    iterable of (start, nbytes, name); empty ranges are ignored."""
    live = sorted((int(a), int(a) + int(n), name) for a, n, name in spans if int(n) > 0)
    for (a0, e0, n0), (a1, _, n1) in zip(live, live[1:]):
        if a1 < e0:
            raise ValueError(f"{n0} and {n1} share memory; every buffer of the step "
                             "must be disjoint from the others")


def _extent(t, name):
    """(start, nbytes, name) of the memory a strided tensor spans."""
    if t.numel() == 0:
        return (t.data_ptr(), 0, name)
    last = sum((size - 1) * stride for size, stride in zip(t.shape, t.stride()))
    return (t.data_ptr(), (last + 1) * t.element_size(), name)


def workspace_bytes(numels):
    """Workspace bytes for a list of tensors with these element counts."""
    return _abi.asr_adamw_workspace_bytes([dict(numel=int(n)) for n in numels])


def make_workspace(numels, device):
    """A device buffer big enough for a list of tensors with these numels."""
    return torch.empty(max(workspace_bytes(numels), 1), dtype=torch.uint8, device=device)


_STEP_NAMES = ("param", "grad", "exp_avg", "exp_avg_sq")
_SMALL_LIST = 8   # lists up to this long take the plain overlap check (less fixed cost)
_ELEM_BYTES = {torch.float32: 4, torch.bfloat16: 2}


def _step_descriptors(params, grads, exp_avgs, exp_avg_sqs, base_indices, device):
    """Checks the four lists and returns their asr_tensor array (numpy), its
    address and the workspace bytes the step needs. Raises TypeError /
    ValueError."""
    n = len(params)
    lists = (params, grads, exp_avgs, exp_avg_sqs)
    index = device.index
    for ts, name in zip(lists, _STEP_NAMES):
        for i, t in enumerate(ts):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name}[{i}] must be a torch.Tensor")
            if not t.is_cuda:
                raise ValueError(f"{name}[{i}] must be on a GPU (got {t.device})")
            if t.get_device() != index:
                raise ValueError("all tensors must be on one device")
            if not t.is_contiguous():
                raise ValueError(f"{name}[{i}] must be contiguous")
    pdt, gdt = [p.dtype for p in params], [g.dtype for g in grads]
    for i, (a, b) in enumerate(zip(pdt, gdt)):
        if a not in _DTYPE_CODE or b not in _DTYPE_CODE:
            raise TypeError(f"tensor {i}: params and grads must be float32 or bfloat16")
    for ts in (exp_avgs, exp_avg_sqs):
        for i, t in enumerate(ts):
            if t.dtype != torch.float32:
                raise TypeError(f"tensor {i}: optimizer states must be float32")
    numels = [p.numel() for p in params]
    for ts in lists[1:]:
        for i, (t, k) in enumerate(zip(ts, numels)):
            if t.numel() != k:
                raise ValueError(f"tensor {i}: param, grad and states differ in size")
    arr = np.zeros(n, dtype=_abi.ASR_TENSOR_DTYPE)
    ptrs = [[t.data_ptr() for t in ts] for ts in lists]
    for name, col in zip(_STEP_NAMES, ptrs):
        arr[name] = col
    arr["numel"] = numels
    arr["base_index"] = [_u64(f"base_indices[{i}]", b) for i, b in enumerate(base_indices)]
    arr["param_dtype"] = [_DTYPE_CODE[d] for d in pdt]
    arr["grad_dtype"] = [_DTYPE_CODE[d] for d in gdt]
    # p, m and v are written in place, so no buffer may share memory with another
    if n <= _SMALL_LIST:
        sizes = [[k * _ELEM_BYTES[d] for k, d in zip(numels, pdt)],
                 [k * _ELEM_BYTES[d] for k, d in zip(numels, gdt)],
                 [k * 4 for k in numels], [k * 4 for k in numels]]
        check_disjoint((a, b, f"{name}[{i}]")
                       for name, col, sz in zip(_STEP_NAMES, ptrs, sizes)
                       for i, (a, b) in enumerate(zip(col, sz)))
    else:
        num = np.asarray(numels, dtype=np.int64)
        sizes = [num * np.asarray([_ELEM_BYTES[d] for d in pdt], dtype=np.int64),
                 num * np.asarray([_ELEM_BYTES[d] for d in gdt], dtype=np.int64), num * 4, num * 4]
        starts = np.concatenate([np.asarray(c, dtype=np.uint64) for c in ptrs])
        _check_disjoint_arrays(starts, np.concatenate(sizes).astype(np.uint64),
                               lambda k: f"{_STEP_NAMES[k // n]}[{k % n}]")
    address = _abi.array_address(arr)
    return arr, address, _abi.asr_adamw_workspace_bytes_at(address, n)


def _check_disjoint_arrays(starts, nbytes, name_of):
    """check_disjoint over arrays of starts and sizes (uint64); name_of(k)
    names span k in the error."""
    live = np.nonzero(nbytes > 0)[0]
    if live.size < 2:
        return
    order = live[np.argsort(starts[live], kind="stable")]
    ends = starts[order] + nbytes[order]
    bad = np.nonzero(starts[order[1:]] < ends[:-1])[0]
    if bad.size:
        k0, k1 = int(order[bad[0]]), int(order[bad[0] + 1])
        raise ValueError(f"{name_of(k0)} and {name_of(k1)} share memory; every buffer of the "
                         "step must be disjoint from the others")


def _step_key(params, grads, exp_avgs, exp_avg_sqs, base_indices, device):
    """What the descriptors of a list depend on: addresses, sizes, dtypes,
    base indices and the device."""
    return (device, tuple(p.data_ptr() for p in params), tuple(g.data_ptr() for g in grads),
            tuple(m.data_ptr() for m in exp_avgs), tuple(v.data_ptr() for v in exp_avg_sqs),
            tuple(p.numel() for p in params), tuple(p.dtype for p in params),
            tuple(g.dtype for g in grads), tuple(base_indices))


def adamw_step(params, grads, exp_avgs, exp_avg_sqs, base_indices, *, lr, beta1, beta2,
               eps, weight_decay, step, seed, rounding="sr", workspace=None, _cache=None):
    """One fused AdamW step over lists of tensors on one device (in place).

    params: f32 or bf16; grads: f32 or bf16, same numel as their param;
    exp_avgs / exp_avg_sqs: f32; base_indices: global position of element 0
    of each tensor. ``rounding`` ("sr" | "rn") applies to bf16 params.

    ``_cache`` (internal, for AdamWSR): a dict kept across steps of one
    list. The checked descriptor array is kept in it and reused while every
    tensor keeps its address, size and dtype and the base indices stay the
    same; anything else is checked again. Contiguity and the device are
    checked only then, so the caller must keep its tensors contiguous and on
    one device (AdamWSR checks its parameters and grads at every step).
    """
    n = len(params)
    if not (len(grads) == len(exp_avgs) == len(exp_avg_sqs) == len(base_indices) == n):
        raise ValueError("all lists must have the same length")
    if rounding not in ROUNDING_CODE:
        raise ValueError("rounding must be 'sr' or 'rn'")
    seed = _u32("seed", seed)
    step = operator.index(step)
    if not 1 <= step < (1 << 32):
        raise ValueError("step must be in [1, 2**32 - 1]")
    if n == 0:
        return
    if not isinstance(params[0], torch.Tensor):
        raise TypeError("param[0] must be a torch.Tensor")
    device = params[0].device
    if device.type != "cuda":
        raise ValueError(f"param[0] must be on a GPU (got {device})")
    if _cache is not None:
        try:
            key = _step_key(params, grads, exp_avgs, exp_avg_sqs, base_indices, device)
        except (AttributeError, TypeError):   # not all tensors: the full check says why
            key = None
        if key is None or _cache.get("key") != key:
            _cache.clear()
            arr, address, need = _step_descriptors(params, grads, exp_avgs, exp_avg_sqs,
                                                   base_indices, device)
            if key is not None:   # (the array stays alive in the cache with its address)
                _cache.update(key=key, arr=arr, address=address, need=need)
        else:
            arr, address, need = _cache["arr"], _cache["address"], _cache["need"]
    else:
        arr, address, need = _step_descriptors(params, grads, exp_avgs, exp_avg_sqs,
                                               base_indices, device)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    if workspace.device != device or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must be on {device} and hold {need} bytes")
    with torch.cuda.device(device):
        _abi.asr_adamw_step_at(address, n, float(lr), float(beta1), float(beta2), float(eps),
                               float(weight_decay), step, seed, ROUNDING_CODE[rounding],
                               workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                               _stream(device))
    _written([*params, *exp_avgs, *exp_avg_sqs])


def philox_4x32_fill(n_counters, counter_base, seed, step, counter_upper=0, *, out=None,
                     device="cuda"):
    """Words of n_counters Philox4x32-10 calls as an int32 tensor of 4*n_counters
    (reinterpret as uint32)."""
    args = (_u64("counter_base", counter_base), _u64("counter_upper", counter_upper),
            _u32("seed", seed), _u32("step", step))
    if out is None:
        out = torch.empty(4 * n_counters, dtype=torch.int32, device=device)
    _require_gpu(out, "out")
    if out.dtype != torch.int32 or out.numel() != 4 * n_counters:
        raise ValueError("out must be int32 with 4*n_counters elements")
    with torch.cuda.device(out.device):
        _abi.asr_philox_4x32_fill(out.data_ptr(), n_counters, *args, _stream(out.device))
    _written(out)
    return out


def _convert_args(x, out):
    _require_gpu(x, "x")
    if x.dtype != torch.float32:
        raise TypeError("x must be float32")
    if out is None:
        out = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    _require_gpu(out, "out")
    if out.dtype != torch.bfloat16 or out.numel() != x.numel() or out.device != x.device:
        raise ValueError("out must be bfloat16 with x's size, on x's device")
    check_disjoint([_extent(x, "x"), _extent(out, "out")])
    return out


def cvt_f32_bf16_sr(x, seed, step, base_index=0, *, out=None):
    """Stochastic rounding f32 -> bf16 (element i at position base_index + i)."""
    key = (_u32("seed", seed), _u32("step", step), _u64("base_index", base_index))
    out = _convert_args(x, out)
    with torch.cuda.device(x.device):
        _abi.asr_cvt_f32_bf16_sr(x.data_ptr(), out.data_ptr(), x.numel(), *key, _stream(x.device))
    _written(out)
    return out


def cvt_f32_bf16_rn(x, *, out=None):
    """Round-to-nearest-even f32 -> bf16."""
    out = _convert_args(x, out)
    with torch.cuda.device(x.device):
        _abi.asr_cvt_f32_bf16_rn(x.data_ptr(), out.data_ptr(), x.numel(), _stream(x.device))
    _written(out)
    return out


def gemm_bf16(a, b, *, rounding="rn", seed=0, step=0, base_index=0, out=None, out_f32=None):
    """C = A B^T for bf16 A (M x K) and B (N x K), rounded to bf16.

    rounding "rn" (round to nearest even) or "sr" (stochastic: element
    (m, n) uses stream position base_index + m*N + n under key (seed,
    step)). ``out``: optional bf16 (M x N) destination, row stride >= N;
    ``out_f32``: optional float32 (M x N) tensor with the same strides as
    ``out`` that also receives the unrounded result. Returns ``out``.
    """
    if rounding not in ("rn", "sr"):
        raise ValueError("rounding must be 'rn' or 'sr'")
    key = (_u32("seed", seed), _u32("step", step), _u64("base_index", base_index))
    for t, name in ((a, "a"), (b, "b")):
        _require_gpu(t, name)
        if t.dtype != torch.bfloat16 or t.dim() != 2:
            raise TypeError(f"{name} must be a 2-D bfloat16 tensor")
        if t.stride(1) != 1:
            raise ValueError(f"{name} must have unit stride along K")
    if a.device != b.device:
        raise ValueError("a and b must be on the same device")
    if a.shape[1] != b.shape[1]:
        raise ValueError(f"K mismatch: a is {tuple(a.shape)}, b is {tuple(b.shape)}")
    m, k = a.shape
    n = b.shape[0]
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=a.device)
    if out.dtype != torch.bfloat16 or tuple(out.shape) != (m, n) or out.device != a.device \
            or (m > 0 and n > 0 and out.stride(1) != 1):
        raise ValueError("out must be a bfloat16 (M, N) tensor with unit column stride")
    ldc = out.stride(0) if m > 1 else max(n, 1)
    f32_ptr = None
    if out_f32 is not None:
        if out_f32.dtype != torch.float32 or tuple(out_f32.shape) != (m, n) \
                or out_f32.device != a.device or out_f32.stride() != out.stride():
            raise ValueError("out_f32 must be a float32 (M, N) tensor with out's strides")
        f32_ptr = out_f32.data_ptr()
    outputs = [_extent(out, "out")] + ([_extent(out_f32, "out_f32")] if out_f32 is not None else [])
    check_disjoint(outputs)
    for o in outputs:
        for i in (_extent(a, "a"), _extent(b, "b")):
            check_disjoint([o, i])
    # a row stride only matters when there is a second row and a K to walk
    lda = a.stride(0) if m > 1 and k > 0 else max(k, 8)
    ldb = b.stride(0) if n > 1 and k > 0 else max(k, 8)
    code = ASR_ROUND_SR if rounding == "sr" else ASR_ROUND_RN
    with torch.cuda.device(a.device):
        _abi.asr_gemm_bf16(a.data_ptr(), lda, b.data_ptr(), ldb, out.data_ptr(), ldc, f32_ptr,
                           m, n, k, code, *key, _stream(a.device))
    _written([out] if out_f32 is None else [out, out_f32])
    return out


def _require_matrix(t, name, dtypes):
    """t is a 2-D GPU tensor of one of `dtypes` whose rows are contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU (got {t.device})")
    if t.dtype not in dtypes or t.dim() != 2:
        raise TypeError(f"{name} must be a 2-D tensor of " +
                        " or ".join(str(d).replace("torch.", "") for d in dtypes))
    if not t.is_contiguous() and t.numel() > 0:
        if t.shape[1] > 1 and t.stride(1) != 1:
            raise ValueError(f"{name} must have unit stride along its rows")
        if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
            raise ValueError(f"{name}: rows must not overlap")


def _row_stride(t, least):
    """Row stride of t, or `least` where there is no second row to walk to."""
    rows, cols = t.shape
    return t.stride(0) if rows > 1 and cols > 0 else max(least, 1)


def _padded16(n):
    return (n + 15) // 16 * 16


def _key(seed, step, base_index):
    if type(seed) is type(step) is type(base_index) is int and 0 <= seed < 1 << 32 \
            and 0 <= step < 1 << 32 and 0 <= base_index < 1 << 64:
        return seed, step, base_index
    return _u32("seed", seed), _u32("step", step), _u64("base_index", base_index)


def quantize_i8(x, *, transpose=False, rounding="rn", seed=0, step=0, base_index=0):
    """8-bit codes of a float32 or bfloat16 matrix: (q, scale).

    One scale a row, ``scale = max|x| / 127``: q is (R, C) int8 and
    x is about ``q * scale[:, None]``. ``transpose=True``: one scale a COLUMN
    of x, and q is the codes of x^T, (C, R) -- the operand of a product that
    sums over x's rows. rounding "rn" (nearest, ties to even) or "sr"
    (stochastic: x's element (i, j) uses stream position base_index + i*C +
    j under key (seed, step), transposed or not). A row with an Inf or NaN
    has scale NaN; one of zeros has scale 0.

    q is a view of rows padded to a multiple of 16 bytes with zeros, which
    ``gemm_i8`` takes as it is. x may have any row stride >= C.
    """
    if rounding not in ROUNDING_CODE:
        raise ValueError("rounding must be 'rn' or 'sr'")
    key = _key(seed, step, base_index)
    _require_matrix(x, "x", (torch.float32, torch.bfloat16))
    rows, cols = x.shape
    device = x.device
    groups, length = (cols, rows) if transpose else (rows, cols)
    ldq = max(_padded16(length), 16)
    store = torch.empty((groups, ldq), dtype=torch.int8, device=device)
    scale = torch.empty(groups, dtype=torch.float32, device=device)
    workspace, need = None, 0
    if transpose:
        need = _abi.asr_quantize_i8_workspace_bytes(rows, cols, 1)
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    with _on(device):
        _abi.asr_quantize_i8(x.data_ptr(), _DTYPE_CODE[x.dtype], _row_stride(x, cols), rows, cols,
                             1 if transpose else 0, store.data_ptr(), ldq, scale.data_ptr(),
                             ROUNDING_CODE[rounding], *key,
                             workspace.data_ptr() if need else None, need, _stream(device))
    return (store if ldq == length else store[:, :length]), scale


def gemm_i8(a, b, scale_a, scale_b, *, rounding="rn", seed=0, step=0, base_index=0, out=None,
            out_f32=None):
    """C = round((A B^T * scale_a[:, None]) * scale_b), rounded to bf16.

    a (M x K) and b (N x K): int8, unit stride along K, row strides multiples
    of 16 and 16-byte aligned starts (as ``quantize_i8`` lays them out); K
    below 2**17, the sums exact integers. scale_a (M) and scale_b (N): float32.
    Rounding, keys, ``out`` and ``out_f32`` as in ``gemm_bf16``.
    """
    if rounding not in ROUNDING_CODE:
        raise ValueError("rounding must be 'rn' or 'sr'")
    key = _key(seed, step, base_index)
    _require_matrix(a, "a", (torch.int8,))
    _require_matrix(b, "b", (torch.int8,))
    device = a.device
    if b.device != device:
        raise ValueError("a and b must be on the same device")
    (m, k), (n, kb) = a.shape, b.shape
    if k != kb:
        raise ValueError(f"K mismatch: a is {tuple(a.shape)}, b is {tuple(b.shape)}")
    for t, size, name in ((scale_a, m, "scale_a"), (scale_b, n, "scale_b")):
        _require_gpu(t, name)
        if t.dtype != torch.float32 or t.dim() != 1 or t.shape[0] != size or t.device != device:
            raise ValueError(f"{name} must be a float32 tensor of shape ({size},) on a's device")
    f32_ptr, given = None, [t for t in (out, out_f32) if t is not None]
    if not given:
        out, ldc = torch.empty((m, n), dtype=torch.bfloat16, device=device), max(n, 1)
    else:   # caller's memory: it may not be what the product reads
        if out is None:
            out = torch.empty((m, n), dtype=torch.bfloat16, device=device)
        _require_matrix(out, "out", (torch.bfloat16,))
        if tuple(out.shape) != (m, n) or out.device != device:
            raise ValueError("out must be a bfloat16 (M, N) tensor on a's device")
        ldc, outputs = _row_stride(out, n), [_extent(out, "out")]
        if out_f32 is not None:
            if out_f32.dtype != torch.float32 or tuple(out_f32.shape) != (m, n) \
                    or out_f32.device != device or out_f32.stride() != out.stride():
                raise ValueError("out_f32 must be a float32 (M, N) tensor with out's strides")
            f32_ptr = out_f32.data_ptr()
            outputs.append(_extent(out_f32, "out_f32"))
        check_disjoint(outputs)
        for o in outputs:
            for t, name in ((a, "a"), (b, "b"), (scale_a, "scale_a"), (scale_b, "scale_b")):
                check_disjoint([o, _extent(t, name)])
    ldk = max(_padded16(k), 16)
    with _on(device):
        _abi.asr_gemm_i8(a.data_ptr(), _row_stride(a, ldk), b.data_ptr(), _row_stride(b, ldk),
                         scale_a.data_ptr(), scale_b.data_ptr(), out.data_ptr(), ldc, f32_ptr, m,
                         n, k, ROUNDING_CODE[rounding], *key, _stream(device))
    if given:
        _written(given)
    return out


NS_COEFFICIENTS = (3.4445, -4.7750, 2.0315)
MUON_MAX_SIDE = 1 << 20


def _coefficients(c):
    c = tuple(float(x) for x in c)
    if len(c) != 3:
        raise ValueError("three Newton-Schulz coefficients (a, b, c) are needed")
    return c


def _ns_workspace(workspace, need, device, spans):
    """The caller's workspace, checked against the buffers at `spans`, or one
    of torch's for this call and stream (its own in every captured graph)."""
    if workspace is None:
        return torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    _require_gpu(workspace, "workspace")
    check_disjoint([*spans, _extent(workspace, "workspace")])
    if workspace.device != device or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must be on {device} and hold {need} bytes")
    return workspace


def newton_schulz(g, *, steps=5, coefficients=NS_COEFFICIENTS, eps=1e-7, out=None, workspace=None):
    """Orthogonalises a matrix, or each of a batch, by Newton-Schulz products.

    g: float32 or bfloat16, (M, N) or (B, M, N), contiguous. X = g / (|g|_F +
    eps), then ``steps`` times X = a X + (b A + c A A) X with A = X X^T (on
    the short side); the result is bfloat16 (nearest even) of g's shape.
    f16 products with f32 sums, X held as two f16 numbers, so the result is off
    the exact one (relative, Frobenius norm, its bf16 rounding apart) by up to
    3e-3 for entries of varied size and a short side of 64 or more, 4e-3 for one
    of 16 to 63, and 1.8e-2 where few or equal roundings do not average: shorter
    sides, entries of one magnitude, orthogonal rows, a single entry. A norm below
    1e-5 eps falls under f16's range: up to 4.1e-5 off in all. A g of zeros gives
    zeros, a matrix with an Inf or NaN only NaN. ``out``: bfloat16, g's shape,
    contiguous (g itself if it is bfloat16).
    """
    coefficients = _coefficients(coefficients)
    _require_gpu(g, "g")
    if g.dtype not in _DTYPE_CODE or g.dim() not in (2, 3):
        raise TypeError("g must be a float32 or bfloat16 tensor of 2 or 3 dimensions")
    if out is None:
        out = torch.empty(g.shape, dtype=torch.bfloat16, device=g.device)
    else:
        _require_gpu(out, "out")
        if out.dtype != torch.bfloat16 or out.shape != g.shape or out.device != g.device:
            raise ValueError("out must be bfloat16 with g's shape, on g's device")
        if out.data_ptr() != g.data_ptr() or g.dtype != torch.bfloat16:
            check_disjoint([_extent(g, "g"), _extent(out, "out")])
    spans = [_extent(g, "g")] + ([_extent(out, "out")] if out.data_ptr() != g.data_ptr() else [])
    rows, cols = g.shape[-2:]
    n = g.shape[0] if g.dim() == 3 else 1
    need = _abi.asr_newton_schulz_workspace_bytes(n, rows, cols)
    workspace = _ns_workspace(workspace, need, g.device, spans)
    size, size_out = rows * cols * g.element_size(), rows * cols * 2
    with _on(g.device):
        _abi.asr_newton_schulz([g.data_ptr() + k * size for k in range(n)],
                               [out.data_ptr() + k * size_out for k in range(n)], rows, cols,
                               _DTYPE_CODE[g.dtype], operator.index(steps), *coefficients,
                               float(eps), workspace.data_ptr(),
                               workspace.numel() * workspace.element_size(), _stream(g.device))
    _written(out)
    return out


def muon_lr_factor(rows, cols, adjust_lr="original"):
    """What Muon multiplies the learning rate of a (rows, cols) matrix by:
    "original" sqrt(max(1, rows / cols)), or "match_rms_adamw" 0.2
    sqrt(max(rows, cols)) (updates as large as AdamW's)."""
    if adjust_lr == "original":
        return max(1.0, rows / cols) ** 0.5 if cols else 1.0
    if adjust_lr == "match_rms_adamw":
        return 0.2 * max(rows, cols) ** 0.5
    raise ValueError("adjust_lr must be 'original' or 'match_rms_adamw'")


def muon_workspace_bytes(shapes):
    """Workspace bytes that hold a muon_step over matrices of these shapes, all
    of one type of param and grad (of several: the largest of each one's)."""
    arr = _abi.muon_array([(None, None, None, r, c, 0, 1.0) for r, c in shapes])
    return _abi.asr_muon_workspace_bytes(arr, len(shapes))


def muon_step(params, grads, momenta, base_indices, *, lr, momentum=0.95, nesterov=True,
              weight_decay=0.0, ns_steps=5, ns_coefficients=NS_COEFFICIENTS, eps=1e-7,
              adjust_lr="original", step, seed, rounding="sr", workspace=None):
    """One Muon step over lists of matrices on one device (in place).

    params: 2-D, f32 or bf16; grads: f32 or bf16; momenta: f32; all
    contiguous, of one shape a matrix. m = momentum*m + g, u = g + momentum*m
    (nesterov) or m, p = p*(1 - lr*weight_decay) - lr*factor*newton_schulz(u),
    with factor = muon_lr_factor(rows, cols, adjust_lr). bf16 params are
    rounded by ``rounding`` ("sr": element i of a matrix at position
    base_index + i under key (seed, step), or "rn"). Matrices of one type go
    through the products together, whatever their shapes.
    """
    n = len(params)
    if not (len(grads) == len(momenta) == len(base_indices) == n):
        raise ValueError("all lists must have the same length")
    if rounding not in ROUNDING_CODE:
        raise ValueError("rounding must be 'sr' or 'rn'")
    seed = _u32("seed", seed)
    step = operator.index(step)
    if not 1 <= step < (1 << 32):
        raise ValueError("step must be in [1, 2**32 - 1]")
    coefficients = _coefficients(ns_coefficients)
    muon_lr_factor(1, 1, adjust_lr)
    groups, spans, device = {}, [], None
    for i, (p, g, m, base) in enumerate(zip(params, grads, momenta, base_indices)):
        for t, name in ((p, "param"), (g, "grad"), (m, "momentum")):
            _require_gpu(t, f"{name}[{i}]")
            device = device or t.device
            if t.device != device:
                raise ValueError("all tensors must be on one device")
            spans.append((t.data_ptr(), t.numel() * t.element_size(), f"{name}[{i}]"))
        if p.dtype not in _DTYPE_CODE or g.dtype not in _DTYPE_CODE or p.dim() != 2:
            raise TypeError(f"matrix {i}: params and grads must be 2-D float32 or bfloat16")
        if m.dtype != torch.float32:
            raise TypeError(f"matrix {i}: momenta must be float32")
        if g.shape != p.shape or m.shape != p.shape:
            raise ValueError(f"matrix {i}: param, grad and momentum differ in shape")
        rows, cols = p.shape
        # (the library's own limit, here for all types' lists before the first is launched)
        if max(rows, cols) > MUON_MAX_SIDE:
            raise ValueError(f"matrix {i}: sides must be at most 2**20")
        groups.setdefault((p.dtype, g.dtype), []).append(
            (p.data_ptr(), g.data_ptr(), m.data_ptr(), rows, cols,
             _u64(f"base_indices[{i}]", base), muon_lr_factor(rows, cols, adjust_lr)))
    if n == 0:
        return
    check_disjoint(spans)
    groups = {key: (_abi.muon_array(ts), len(ts)) for key, ts in groups.items()}
    need = max(_abi.asr_muon_workspace_bytes(arr, k) for arr, k in groups.values())
    workspace = _ns_workspace(workspace, need, device, spans)
    with _on(device):
        for (pt, gt), (arr, k) in groups.items():
            _abi.asr_muon_step(arr, k, _DTYPE_CODE[pt], _DTYPE_CODE[gt], float(lr),
                               float(momentum), int(bool(nesterov)), float(weight_decay),
                               operator.index(ns_steps), coefficients, float(eps), step, seed,
                               ROUNDING_CODE[rounding], workspace.data_ptr(),
                               workspace.numel() * workspace.element_size(), _stream(device))
    _written([*params, *momenta])


class RoundingMode:
    """Rounding modes of the f32 -> bf16 conversion ("Add stochastic rounding
    and philox RNG helpers", discussion: stochastic rounding as a rounding
    mode of the existing conversion, keyed by a seed)."""
    NEAREST = "rn"
    STOCHASTIC = "sr"


def to(x, dtype=torch.bfloat16, *, rounding=RoundingMode.NEAREST, seed=0, step=0, base_index=0,
       out=None):
    """x.to(dtype) with a choice of rounding, for float32 -> bfloat16.

    rounding NEAREST: round to nearest even. STOCHASTIC: element i uses the
    16 random bits of stream position base_index + i under key (seed, step)
    (asr_cvt_f32_bf16_sr). Any shape; x must be contiguous float32 on a GPU.
    A float32 -> float32 request returns x itself.
    """
    if dtype == x.dtype == torch.float32:
        return x
    if dtype != torch.bfloat16:
        raise NotImplementedError("to(): float32 -> bfloat16 only")
    if rounding in (RoundingMode.STOCHASTIC, "sr", "stochastic"):
        return cvt_f32_bf16_sr(x, seed, step, base_index, out=out)
    if rounding in (RoundingMode.NEAREST, "rn", "nearest"):
        return cvt_f32_bf16_rn(x, out=out)
    raise ValueError(f"unknown rounding {rounding!r}")


def f32_sqrt_div(a, b):
    """(sqrt(a), a / b) as the AdamW kernel evaluates them (test support)."""
    for t, name in ((a, "a"), (b, "b")):
        _require_gpu(t, name)
        if t.dtype != torch.float32:
            raise TypeError(f"{name} must be float32")
    if a.numel() != b.numel() or a.device != b.device:
        raise ValueError("a and b must match in size and device")
    s = torch.empty_like(a)
    d = torch.empty_like(a)
    with torch.cuda.device(a.device):
        _abi.asr_f32_sqrt_div(a.data_ptr(), b.data_ptr(), s.data_ptr(), d.data_ptr(), a.numel(),
                              _stream(a.device))
    return s, d


def sr_bf16_given_bits(x, r16, *, out=None):
    """SR f32 -> bf16 with caller-supplied random bits r16 (int16 tensor whose
    bit patterns are the 16-bit random values)."""
    _require_gpu(x, "x")
    _require_gpu(r16, "r16")
    if x.dtype != torch.float32 or r16.dtype != torch.int16 or r16.numel() != x.numel():
        raise ValueError("x must be float32 and r16 int16 of the same size")
    out = _convert_args(x, out)
    check_disjoint([_extent(r16, "r16"), _extent(out, "out")])
    with torch.cuda.device(x.device):
        _abi.asr_sr_bf16_given_bits(x.data_ptr(), r16.data_ptr(), out.data_ptr(), x.numel(),
                                    _stream(x.device))
    _written(out)
    return out
