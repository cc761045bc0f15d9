"""Refusals of the int8 entry points (CPU only; no call here launches a kernel)."""

import pytest
import torch

from adamw_optimizer_stochastic_amd import _abi, _build, linear_i8, ops


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


def test_quantize_argument_errors():
    E = _abi

    def q(x=0x1000, dtype=E.ASR_BF16, ldx=64, rows=8, cols=60, transpose=0, q=0x4000, ldq=64,
          scale=0x8000, rounding=E.ASR_ROUND_SR, base=0, ws=None, ws_bytes=0):
        return _status(E.asr_quantize_i8, x, dtype, ldx, rows, cols, transpose, q, ldq, scale,
                       rounding, 1, 2, base, ws, ws_bytes, None)

    assert q(rows=-1) == E.ASR_EINVAL
    assert q(cols=2 ** 31) == E.ASR_EINVAL
    assert q(dtype=2) == E.ASR_EDTYPE
    assert q(rounding=3) == E.ASR_EINVAL
    assert q(x=0) == E.ASR_EINVAL
    assert q(q=0) == E.ASR_EINVAL
    assert q(scale=0) == E.ASR_EINVAL
    assert q(ldx=59) == E.ASR_EINVAL
    assert q(ldq=48) == E.ASR_EINVAL
    assert q(ldq=72) == E.ASR_EINVAL
    assert q(x=0x1001) == E.ASR_EALIGN
    assert q(dtype=E.ASR_F32, x=0x1002) == E.ASR_EALIGN
    assert q(q=0x4008) == E.ASR_EALIGN
    assert q(scale=0x8002) == E.ASR_EALIGN
    assert q(base=2 ** 64 - 8 * 60 + 1) == E.ASR_EINVAL
    assert q(transpose=1, ldq=16) == E.ASR_EWORKSPACE
    need = E.asr_quantize_i8_workspace_bytes(8, 60, 1)
    assert need >= 60 * 4 and E.asr_quantize_i8_workspace_bytes(8, 60, 0) == 0
    assert q(transpose=1, ldq=16, ws=0x10000, ws_bytes=need - 1) == E.ASR_EWORKSPACE
    assert q(transpose=1, ldq=16, ws=0x10008, ws_bytes=need) == E.ASR_EWORKSPACE
    assert q(rows=2 ** 26) == E.ASR_EINVAL          # 2**24 workgroups of four rows
    assert q(rows=2 ** 24, cols=4096, ldx=4096, ldq=4096) == E.ASR_EINVAL
    assert q(transpose=1, rows=2 ** 29, cols=2 ** 20, ldx=2 ** 20, ldq=2 ** 29, ws=0x10000,
             ws_bytes=1 << 50) == E.ASR_EINVAL
    assert q(rows=0, x=0, q=0, scale=0) == E.ASR_OK
    assert q(cols=0, transpose=1, x=0, q=0, scale=0) == E.ASR_OK


def test_gemm_i8_argument_errors():
    E = _abi

    def g(a=0x1000, lda=64, b=0x2000, ldb=64, sa=0x5000, sb=0x6000, c=0x3000, ldc=32, c32=None,
          m=16, n=32, k=60, rounding=E.ASR_ROUND_SR, base=0):
        return _status(E.asr_gemm_i8, a, lda, b, ldb, sa, sb, c, ldc, c32, m, n, k, rounding, 1,
                       2, base, None)

    assert g(m=-1) == E.ASR_EINVAL
    assert g(n=2 ** 31) == E.ASR_EINVAL
    assert g(k=2 ** 17, lda=2 ** 17, ldb=2 ** 17) == E.ASR_EINVAL
    assert g(rounding=2) == E.ASR_EINVAL
    for name in ("a", "b", "sa", "sb", "c"):
        assert g(**{name: 0}) == E.ASR_EINVAL
    assert g(lda=48) == E.ASR_EINVAL
    assert g(ldc=31) == E.ASR_EINVAL
    assert g(lda=2 ** 23) == E.ASR_EINVAL
    assert g(ldb=72) == E.ASR_EALIGN
    assert g(a=0x1008) == E.ASR_EALIGN
    assert g(c=0x3001) == E.ASR_EALIGN
    assert g(c32=0x3002) == E.ASR_EALIGN
    assert g(sa=0x5001) == E.ASR_EALIGN
    assert g(base=2 ** 64 - 16 * 32 + 1) == E.ASR_EINVAL
    assert g(m=0, a=0, b=0, c=0, sa=0, sb=0) == E.ASR_OK


def test_binding_refuses_what_is_not_on_a_gpu():
    x = torch.zeros(4, 16)
    q = torch.zeros(4, 16, dtype=torch.int8)
    s = torch.zeros(4)
    w = torch.zeros(4, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        ops.quantize_i8(x)
    with pytest.raises(ValueError, match="GPU"):
        ops.gemm_i8(q, q, s, s)
    with pytest.raises(ValueError, match="GPU"):
        linear_i8(w, w)
    with pytest.raises(ValueError, match="rounding"):
        ops.quantize_i8(x, rounding="up")
    with pytest.raises(ValueError, match="rounding"):
        linear_i8(w, w, grad_rounding="up")
    with pytest.raises(TypeError):
        ops.quantize_i8([1.0])
    with pytest.raises(TypeError):
        linear_i8(x, w)
    with pytest.raises(ValueError, match="seed"):
        ops.quantize_i8(x, seed=2 ** 32)


def test_linear_argument_errors():
    E = _abi
    need = [E.asr_linear_i8_workspace_bytes(40, 24, 56, b) for b in (0, 1)]
    assert need[0] >= (40 + 24) * 64 and need[1] >= 40 * 32 + 24 * 48 + 56 * 32 + 56 * 48
    for bad in ((-1, 4, 4), (4, 2 ** 17, 4), (0, 4, 4)):
        assert E.asr_linear_i8_workspace_bytes(*bad, 0) == 0

    def fwd(x=0x1000, ldx=56, w=0x8000, ldw=56, y=0x10000, ldy=24, t=40, n=24, k=56, ws=0x100000,
            ws_bytes=need[0]):
        return _status(E.asr_linear_i8_forward, x, ldx, w, ldw, y, ldy, t, n, k, ws, ws_bytes,
                       None)

    assert fwd(t=-1) == E.ASR_EINVAL
    assert fwd(n=2 ** 17) == E.ASR_EINVAL
    assert fwd(k=2 ** 17) == E.ASR_EINVAL
    for name in ("x", "w", "y"):
        assert fwd(**{name: 0}) == E.ASR_EINVAL
        assert fwd(**{name: 0x1001}) == E.ASR_EALIGN
    for name, ld in (("ldx", 55), ("ldw", 55), ("ldy", 23)):
        assert fwd(**{name: ld}) == E.ASR_EINVAL
    assert fwd(ws=0) == E.ASR_EWORKSPACE
    assert fwd(ws=0x100080) == E.ASR_EWORKSPACE
    assert fwd(ws_bytes=need[0] - 1) == E.ASR_EWORKSPACE
    assert fwd(t=0, x=0, y=0, ws=0) == E.ASR_OK

    def bwd(x=0x1000, w=0x8000, dy=0x10000, lddy=24, dx=0x20000, dw=0x30000, t=40, n=24, k=56,
            rounding=E.ASR_ROUND_SR, base=0, ws=0x100000, ws_bytes=need[1]):
        return _status(E.asr_linear_i8_backward, x, 56, w, 56, dy, lddy, dx, 56, dw, 56, t, n, k,
                       rounding, 1, 2, base, ws, ws_bytes, None)

    assert bwd(t=2 ** 17) == E.ASR_EINVAL
    assert bwd(rounding=2) == E.ASR_EINVAL
    for name in ("x", "w", "dy"):
        assert bwd(**{name: 0}) == E.ASR_EINVAL
        assert bwd(**{name: 0x1001}) == E.ASR_EALIGN
    assert bwd(dx=0x20001) == E.ASR_EALIGN
    assert bwd(dw=0x30001) == E.ASR_EALIGN
    assert bwd(lddy=23) == E.ASR_EINVAL
    assert bwd(base=2 ** 64 - 40 * 24 + 1) == E.ASR_EINVAL
    assert bwd(ws=0) == E.ASR_EWORKSPACE
    assert bwd(ws_bytes=need[1] - 1) == E.ASR_EWORKSPACE
    assert bwd(dx=0, dw=0, ws=0) == E.ASR_OK


def test_sizes_past_a_launch_are_refused():
    """Sizes that the arguments' ranges allow and a launch, or a kernel's own
    32-bit counting, does not."""
    E = _abi
    big = 2 ** 31 - 1
    ws = E.asr_quantize_i8_workspace_bytes(big, 1, 1)
    for rows, cols, transpose in ((big, 1, 1), (2 ** 31 - 63, 1, 1), (2 ** 27, 2 ** 12, 1),
                                  (2 ** 24, 4096, 0), (2 ** 26, 1, 0)):
        length = rows if transpose else cols
        assert _status(E.asr_quantize_i8, 0x1000, E.ASR_BF16, cols, rows, cols, transpose, 0x2000,
                       (length + 15) // 16 * 16, 0x3000, E.ASR_ROUND_RN, 0, 0, 0, 0x4000,
                       max(ws, E.asr_quantize_i8_workspace_bytes(rows, cols, 1)), None) \
            == E.ASR_EINVAL
    for m, n in ((5, big), (big, 5), (256, 2 ** 31 - 256 * 256 + 1), (2 ** 30, 2 ** 30)):
        assert _status(E.asr_gemm_i8, 0x1000, 16, 0x2000, 16, 0x3000, 0x4000, 0x5000, n, None, m,
                       n, 16, E.ASR_ROUND_RN, 0, 0, 0, None) == E.ASR_EINVAL
