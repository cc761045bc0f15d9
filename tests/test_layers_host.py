"""Refusals of the layers and of the 8-bit activations (CPU only; no call here
launches a kernel)."""

import pytest
import torch

from adamw_optimizer_stochastic_amd import (_abi, _build, embedding, layer_norm, linear_i8, ops,
                                            silu_mul)

E = _abi


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


def test_pack_argument_errors():
    def p(x=0x1000, dtype=E.ASR_BF16, ldx=64, rows=8, cols=60, q=0x4000, ldq=64, scale=0x8000,
          rounding=E.ASR_ROUND_SR, base=0):
        return _status(E.asr_pack_i8, x, dtype, ldx, rows, cols, q, ldq, scale, rounding, 1, 2,
                       base, None)

    assert p(rows=-1) == E.ASR_EINVAL and p(rows=2 ** 31) == E.ASR_EINVAL
    assert p(cols=2 ** 31 - 4096) == E.ASR_EINVAL
    assert p(dtype=2) == E.ASR_EDTYPE
    assert p(rounding=3) == E.ASR_EINVAL
    for name in ("x", "q", "scale"):
        assert p(**{name: 0}) == E.ASR_EINVAL
    assert p(ldx=59) == E.ASR_EINVAL and p(ldq=48) == E.ASR_EINVAL and p(ldq=72) == E.ASR_EINVAL
    assert p(x=0x1001) == E.ASR_EALIGN and p(q=0x4008) == E.ASR_EALIGN
    assert p(dtype=E.ASR_F32, x=0x1002) == E.ASR_EALIGN and p(scale=0x8002) == E.ASR_EALIGN
    assert p(base=2 ** 64 - 8 * 60 + 1) == E.ASR_EINVAL
    big = 2 ** 31 - 8192
    assert p(rows=2 ** 31 - 1, cols=big, ldx=big, ldq=big) == E.ASR_EINVAL
    assert p(rows=0, x=0, q=0, scale=0) == E.ASR_OK and p(cols=0, x=0, q=0) == E.ASR_OK

    def u(q=0x4000, ldq=64, scale=0x8000, rows=8, cols=60, x=0x1000, dtype=E.ASR_BF16, ldx=64):
        return _status(E.asr_unpack_i8, q, ldq, scale, rows, cols, x, dtype, ldx, None)

    assert u(ldq=56) == E.ASR_EINVAL and u(dtype=7) == E.ASR_EDTYPE and u(ldx=59) == E.ASR_EINVAL
    assert u(q=0) == E.ASR_EINVAL and u(x=0) == E.ASR_EINVAL and u(scale=0) == E.ASR_EINVAL
    assert u(x=0x1001) == E.ASR_EALIGN and u(q=0x4001) == E.ASR_EALIGN
    assert u(rows=0, q=0, x=0, scale=0) == E.ASR_OK


def test_layer_norm_argument_errors():
    def f(x=0x1000, dtype=E.ASR_BF16, ldx=60, rows=8, cols=60, w=0x3000, b=0x4000,
          pdt=E.ASR_BF16, eps=1e-5, y=0x5000, stat=0x8000, q=None, ldq=0, scale=None):
        return _status(E.asr_layer_norm_forward, x, dtype, ldx, rows, cols, w, b, pdt, eps, y,
                       stat, q, ldq, scale, None)

    assert f(rows=-1) == E.ASR_EINVAL and f(rows=2 ** 24) == E.ASR_EINVAL
    assert f(cols=2 ** 24 + 1, ldx=2 ** 25) == E.ASR_EINVAL
    assert f(dtype=5) == E.ASR_EDTYPE and f(pdt=5) == E.ASR_EDTYPE
    for eps in (-1e-9, float("nan"), float("inf")):
        assert f(eps=eps) == E.ASR_EINVAL
    assert f(x=0) == E.ASR_EINVAL and f(y=0) == E.ASR_EINVAL and f(ldx=59) == E.ASR_EINVAL
    assert f(x=0x1001) == E.ASR_EALIGN and f(w=0x3001) == E.ASR_EALIGN
    assert f(b=0x4002, pdt=E.ASR_F32) == E.ASR_EALIGN and f(stat=0x8008) == E.ASR_EALIGN
    assert f(q=0x9000, ldq=64) == E.ASR_EINVAL and f(scale=0x9000, ldq=64) == E.ASR_EINVAL
    assert f(q=0x9000, ldq=60, scale=0xA000) == E.ASR_EINVAL
    assert f(q=0x9004, ldq=64, scale=0xA000) == E.ASR_EALIGN
    assert f(rows=0, x=0, y=0) == E.ASR_OK and f(cols=0, x=0, y=0) == E.ASR_OK

    need = E.asr_layer_norm_backward_workspace_bytes(8, 60)
    assert need == 8 * 2 * 60 * 4
    assert E.asr_layer_norm_backward_workspace_bytes(10 ** 6, 60) == 256 * 2 * 60 * 4
    assert E.asr_layer_norm_backward_workspace_bytes(0, 60) == 0

    def g(dy=0x1000, ld=60, x=0x2000, ldx=60, q=None, ldq=0, scale=None, stat=0x8000,
          dtype=E.ASR_BF16, rows=8, cols=60, w=0x3000, pdt=E.ASR_BF16, dx=0x5000, dw=0x6000,
          db=0x7000, ws=0x10000, ws_bytes=need):
        return _status(E.asr_layer_norm_backward, dy, ld, x, ldx, q, ldq, scale, stat, dtype,
                       rows, cols, w, pdt, dx, dw, db, ws, ws_bytes, None)

    assert g(dy=0) == E.ASR_EINVAL and g(x=0) == E.ASR_EINVAL and g(stat=0) == E.ASR_EINVAL
    assert g(ld=59) == E.ASR_EINVAL and g(ldx=59) == E.ASR_EINVAL
    assert g(q=0x9000, ldq=64, scale=0xA000) == E.ASR_EINVAL       # x as well
    assert g(x=0, q=0x9000, ldq=64) == E.ASR_EINVAL
    assert g(stat=0x8004) == E.ASR_EALIGN and g(dx=0x5001) == E.ASR_EALIGN
    assert g(dw=0x6001) == E.ASR_EALIGN and g(dy=0x1001) == E.ASR_EALIGN
    assert g(ws=0) == E.ASR_EWORKSPACE and g(ws_bytes=need - 1) == E.ASR_EWORKSPACE
    assert g(ws=0x10008) == E.ASR_EWORKSPACE
    assert g(dtype=9) == E.ASR_EDTYPE
    assert g(dx=0, dw=0, db=0, dy=0) == E.ASR_OK
    assert g(rows=0, dw=0, db=0, dy=0, x=0, stat=0) == E.ASR_OK


def test_silu_mul_argument_errors():
    def f(g=0x1000, ldg=120, u=0x1078, ldu=120, dtype=E.ASR_BF16, rows=8, cols=60, y=0x3000,
          ldy=60, qg=None, sg=None, qu=None, su=None, ldq=64):
        return _status(E.asr_silu_mul_forward, g, ldg, u, ldu, dtype, rows, cols, y, ldy, qg, sg,
                       qu, su, ldq, None)

    for name in ("g", "u", "y"):
        assert f(**{name: 0}) == E.ASR_EINVAL and f(**{name: 0x1001}) == E.ASR_EALIGN
    for name in ("ldg", "ldu", "ldy"):
        assert f(**{name: 59}) == E.ASR_EINVAL
    assert f(dtype=3) == E.ASR_EDTYPE and f(rows=2 ** 31) == E.ASR_EINVAL
    codes = dict(qg=0x4000, sg=0x5000, qu=0x6000, su=0x7000)
    for name in codes:
        assert f(**{**codes, name: None}) == E.ASR_EINVAL
    assert f(**codes, ldq=48) == E.ASR_EINVAL and f(**{**codes, "qu": 0x6008}) == E.ASR_EALIGN
    assert f(rows=0, g=0, u=0, y=0) == E.ASR_OK

    def b(dy=0x1000, ldd=60, g=0x2000, ldg=60, u=0x3000, ldu=60, qg=None, sg=None, qu=None,
          su=None, ldq=64, dtype=E.ASR_BF16, rows=8, cols=60, dg=0x4000, lddg=60, du=0x5000,
          lddu=60):
        return _status(E.asr_silu_mul_backward, dy, ldd, g, ldg, u, ldu, qg, sg, qu, su, ldq,
                       dtype, rows, cols, dg, lddg, du, lddu, None)

    for name in ("dy", "g", "u", "dg", "du"):
        assert b(**{name: 0}) == E.ASR_EINVAL and b(**{name: 0x1001}) == E.ASR_EALIGN
    for name in ("ldd", "ldg", "ldu", "lddg", "lddu"):
        assert b(**{name: 59}) == E.ASR_EINVAL
    codes = dict(qg=0x6000, sg=0x7000, qu=0x8000, su=0x9000)
    assert b(**codes) == E.ASR_EINVAL                              # gate and up as well
    assert b(g=0, u=0, **{**codes, "su": None}) == E.ASR_EINVAL
    assert b(rows=0, dy=0, g=0, u=0, dg=0, du=0) == E.ASR_OK


def test_embedding_argument_errors():
    def f(ids=0x1000, wide=1, n=8, table=0x2000, dtype=E.ASR_BF16, ld=60, vocab=100, dim=60,
          scale=1.0, y=0x8000):
        return _status(E.asr_embedding_forward, ids, wide, n, table, dtype, ld, vocab, dim, scale,
                       y, None)

    assert f(n=-1) == E.ASR_EINVAL and f(n=2 ** 31) == E.ASR_EINVAL
    assert f(vocab=2 ** 31) == E.ASR_EINVAL and f(dim=2 ** 24 + 1, ld=2 ** 25) == E.ASR_EINVAL
    assert f(dtype=4) == E.ASR_EDTYPE
    for scale in (float("nan"), float("inf"), 1e39):
        assert f(scale=scale) == E.ASR_EINVAL
    for name in ("ids", "table", "y"):
        assert f(**{name: 0}) == E.ASR_EINVAL and f(**{name: 0x1001}) == E.ASR_EALIGN
    assert f(ids=0x1004) == E.ASR_EALIGN and f(ld=59) == E.ASR_EINVAL
    assert f(n=0, ids=0, table=0, y=0) == E.ASR_OK

    need = E.asr_embedding_backward_workspace_bytes(2000, 100, 60)
    assert need >= 2000 * 8 + 100 // 8 + 125 * 2 * 60 * 4
    assert E.asr_embedding_backward_workspace_bytes(0, 100, 60) == 0
    assert E.asr_embedding_backward_workspace_bytes(8, 100, 60) == 0       # few tokens, small table
    assert E.asr_embedding_backward_workspace_bytes(1024, 1 << 17, 128) == 0
    assert E.asr_embedding_backward_workspace_bytes(1024, (1 << 17) + 1, 128) > 0
    several = E.asr_embedding_backward_workspace_bytes(8193, 100, 60)
    assert several >= 16 * 8193 + 2 * 256 * 4 + 513 * 2 * 60 * 4

    def g(ids=0x1000, wide=1, n=2000, dy=0x2000, ld=60, dtype=E.ASR_BF16, vocab=100, dim=60,
          scale=1.0, padding=-1, dw=0x8000, ws=0x10000, ws_bytes=need):
        return _status(E.asr_embedding_backward, ids, wide, n, dy, ld, dtype, vocab, dim, scale,
                       padding, dw, ws, ws_bytes, None)

    assert g(padding=-2) == E.ASR_EINVAL and g(padding=100) == E.ASR_EINVAL
    for name in ("ids", "dy", "dw"):
        assert g(**{name: 0}) == E.ASR_EINVAL and g(**{name: 0x1001}) == E.ASR_EALIGN
    assert g(ld=59) == E.ASR_EINVAL and g(dtype=4) == E.ASR_EDTYPE
    assert g(ws=0) == E.ASR_EWORKSPACE and g(ws=0x10010) == E.ASR_EWORKSPACE
    assert g(ws_bytes=need - 1) == E.ASR_EWORKSPACE
    assert g(vocab=2 ** 31 - 1, dim=2 ** 24, ld=2 ** 24) == E.ASR_EINVAL
    assert g(vocab=1, n=1 << 14, dim=2 ** 24, ld=2 ** 24) == E.ASR_EINVAL   # the join's workgroups
    assert g(vocab=0, n=0, ids=0, dy=0, dw=0) == E.ASR_OK


def test_linear_saved_argument_errors():
    need = [E.asr_linear_i8_workspace_bytes(40, 24, 56, b) for b in (0, 1)]

    def f(q=0x20000, ldq=64, scale=0x30000, t=40, n=24, k=56):
        return _status(E.asr_linear_i8_forward_saved, 0x1000, 56, 0x8000, 56, 0x10000, 24, q, ldq,
                       scale, t, n, k, None, 0, None)

    assert f() == E.ASR_EWORKSPACE
    assert f(q=0) == E.ASR_EINVAL and f(scale=0) == E.ASR_EINVAL and f(n=0) == E.ASR_EINVAL
    for ldq in (56, 48, 2 ** 23):
        assert f(ldq=ldq) == E.ASR_EINVAL
    assert f(q=0x20008) == E.ASR_EALIGN and f(scale=0x30001) == E.ASR_EALIGN
    assert f(t=2 ** 17) == E.ASR_EINVAL and f(t=0, q=0, scale=0) == E.ASR_OK

    def g(q=0x20000, ldq=64, scale=0x30000, dw=0x40000, dx=0x50000, t=40, n=24, k=56, ws=0,
          ws_bytes=need[1]):
        return _status(E.asr_linear_i8_backward_saved, q, ldq, scale, 0x1000, 56, 0x8000, 24, dx,
                       56, dw, 56, t, n, k, E.ASR_ROUND_SR, 1, 2, 0, ws, ws_bytes, None)

    assert g() == E.ASR_EWORKSPACE
    assert g(q=0) == E.ASR_EINVAL and g(ldq=56) == E.ASR_EINVAL and g(scale=0) == E.ASR_EINVAL
    assert g(q=0x20001) == E.ASR_EALIGN
    assert g(q=0, scale=0, dw=0) == E.ASR_EWORKSPACE              # dx alone needs no codes
    assert g(dw=0, dx=0) == E.ASR_OK and g(k=0, q=0, scale=0) == E.ASR_OK


def test_binding_refusals():
    x, w = torch.zeros(4, 16), torch.zeros(16)
    b = torch.zeros(4, 16, dtype=torch.bfloat16)
    ids = torch.zeros(3, dtype=torch.int64)
    for call in (lambda: ops.pack_i8(x), lambda: layer_norm(x, w, w), lambda: silu_mul(x, x),
                 lambda: embedding(ids, x), lambda: linear_i8(b, b, saved="i8"),
                 lambda: ops.unpack_i8(torch.zeros(4, 16, dtype=torch.int8), torch.zeros(4, 1))):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for call in (lambda: layer_norm(x, saved="x"), lambda: silu_mul(x, saved="input"),
                 lambda: linear_i8(b, b, saved="inputs")):
        with pytest.raises(ValueError, match="saved"):
            call()
    with pytest.raises(ValueError, match="rounding"):
        ops.pack_i8(x, rounding="up")
    with pytest.raises(ValueError, match="seed"):
        ops.pack_i8(x, seed=-1)
    with pytest.raises(TypeError, match="dtype"):
        ops.unpack_i8(x, x, dtype=torch.float16)
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(ValueError, match="eps"):
            layer_norm(x, eps=eps)
    for call in (lambda: layer_norm([1.0]), lambda: silu_mul(None), lambda: embedding(ids, None)):
        with pytest.raises(TypeError):
            call()
