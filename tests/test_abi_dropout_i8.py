"""Host-side tests of the dropout and 8-bit entry points (CPU only: every call
here is refused before anything is launched; the pointers are never read)."""

import ctypes
import math

import pytest

from bit_quantized_finetuning_nf4_amd import _lib, ops
from bit_quantized_finetuning_nf4_amd._lib import DropDesc, I8RowsDesc, Nf4WeightDesc

NULL, ALIGN, SHAPE, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5
P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(12)]
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def ref(x):
    return None if x is None else ctypes.byref(x)


def test_dropout(L):
    d = DropDesc(0.1, 1, 2, None)
    f = lambda x=P[0], n=64, drop=d, y=P[1]: L.qlora_dropout(x, n, ref(drop), y, None)
    assert f(x=None) == NULL and f(y=None) == NULL and f(drop=None) == NULL
    assert f(x=ODD) == ALIGN and f(y=ODD) == ALIGN
    assert f(n=0) == SHAPE and f(n=-1) == SHAPE and f(n=(1 << 36) + 1) == SHAPE
    for p in (-1e-9, 1.0, 7.0, math.nan, math.inf):
        assert f(drop=DropDesc(p, 1, 2, None)) == UNSUPPORTED
    assert f(drop=DropDesc(0.1, 1, 2, 0x10004)) == ALIGN


def test_linear_drop(L):
    w = Nf4WeightDesc(128, 256, 64, 256, P[0].value, P[1].value, P[2].value, 0, 0)
    d = DropDesc(0.1, 1, 2, None)

    def fwd(W=w, X=P[3], M=4, A=P[4], B=P[5], r=8, drop=d, Y=P[6], U=None, ws=P[7], n=1 << 30):
        return L.qlora_linear_fwd_drop(ref(W), X, M, A, B, r, 16.0, ref(drop), Y, U, ws, n, None)

    def bwd(W=w, X=P[3], dY=P[8], M=4, A=P[4], B=P[5], r=8, U=P[9], drop=d, dX=P[6], dA=P[10], dB=P[11], ws=P[7],
            n=1 << 30):
        return L.qlora_linear_bwd_drop(ref(W), X, dY, M, A, B, r, 16.0, U, ref(drop), dX, dA, dB, ws, n, None)

    for f in (fwd, bwd):
        assert f(W=None) == NULL and f(drop=None) == NULL and f(A=None) == NULL and f(X=None) == NULL
        assert f(M=0) == SHAPE and f(r=12) == UNSUPPORTED and f(r=136) == UNSUPPORTED
        assert f(n=16) == WORKSPACE and f(ws=None) == NULL and f(ws=ODD) == ALIGN and f(B=ODD) == ALIGN
        assert f(drop=DropDesc(1.0, 1, 2, None)) == UNSUPPORTED
        assert f(drop=DropDesc(0.5, 1, 2, 0x10004)) == ALIGN
        assert f(W=Nf4WeightDesc(128, 200, 64, 256, P[0].value, P[1].value, P[2].value, 0, 0)) == UNSUPPORTED
        assert f(W=Nf4WeightDesc(132, 256, 64, 256, P[0].value, P[1].value, P[2].value, 0, 0)) == UNSUPPORTED
    assert fwd(r=0, A=None, B=None) == UNSUPPORTED
    assert bwd(r=0, A=None, B=None, dA=None, dB=None) == UNSUPPORTED
    assert bwd(dA=None) == NULL and bwd(dY=None) == NULL and bwd(U=ODD) == ALIGN and bwd(dX=ODD) == ALIGN
    need = L.qlora_workspace_bytes(_lib.QLORA_OP_BWD_DROP, 4, 128, 256, 8, 0)
    assert need >= 128 * 256 * 2 and bwd(n=need - 1) == WORKSPACE


def test_workspace_queries(L):
    q = L.qlora_workspace_bytes
    for op in (_lib.QLORA_OP_BWD_DROP, _lib.QLORA_OP_I8_FWD, _lib.QLORA_OP_I8_BWD):
        assert q(op, 0, 64, 64, 8, 0) == 0 and q(op, 4, 64, 64, -8, 0) == 0 and q(op, 4, 64, 64, 200, 0) == 0
        assert q(op, 4, 64, 1 << 40, 8, 0) == 0
    # a contraction that is not whole 64-column pairs takes padded copies
    assert q(_lib.QLORA_OP_I8_BWD, 100, 72, 64, 8, 0) >= q(_lib.QLORA_OP_I8_BWD, 100, 128, 64, 8, 0) - 4096 + 100 * 128 * 2
    assert q(_lib.QLORA_OP_I8_FWD, 5, 64, 200, 0, 0) >= 5 * 256 + 5 * 4


def test_i8(L):
    rb = L.qlora_i8_row_bytes
    sizes = (-8, 0, 8, 128, 136, 131072, 131080)
    assert [rb(c) for c in sizes] == [ops.i8_row_bytes(c) for c in sizes] == [0, 0, 128, 128, 256, 131072, 0]
    rows = lambda n=64, k=256, c=P[0].value, s=P[1].value: I8RowsDesc(n, k, c, s)
    for call in (lambda q: L.qlora_i8_quantize(P[2], ref(q), None), lambda q: L.qlora_i8_dequant(ref(q), P[2], None),
                 lambda q: L.qlora_i8_matmul(ref(rows(4)), ref(q), P[2], None),
                 lambda q: L.qlora_i8_linear_fwd(ref(q), P[2], 4, None, None, 0, 1.0, None, P[3], None, P[4], 1 << 30, None),
                 lambda q: L.qlora_i8_linear_bwd(ref(q), None, P[2], 4, None, None, 0, 1.0, None, None, P[3], None, None,
                                                 P[4], 1 << 30, None)):
        assert call(None) == NULL and call(rows(0)) == SHAPE and call(rows(k=0)) == SHAPE
        assert call(rows(k=12)) == UNSUPPORTED and call(rows(k=131080)) == UNSUPPORTED
        assert call(rows(n=1 << 24, k=131072)) == UNSUPPORTED
        assert call(rows(c=None)) == NULL and call(rows(s=None)) == NULL
        assert call(rows(c=0x10008)) == ALIGN and call(rows(s=0x10004)) == ALIGN
    assert L.qlora_i8_quantize(None, ref(rows()), None) == NULL
    assert L.qlora_i8_quantize(ODD, ref(rows()), None) == ALIGN
    assert L.qlora_i8_dequant(ref(rows()), None, None) == NULL
    assert L.qlora_i8_matmul(ref(rows(k=128)), ref(rows()), P[2], None) == SHAPE
    assert L.qlora_i8_matmul(ref(rows()), ref(rows(n=60)), P[2], None) == UNSUPPORTED

    def fwd(W=rows(), X=P[2], M=4, A=P[3], B=P[4], r=8, drop=None, Y=P[5], U=None, ws=P[6], n=1 << 30):
        return L.qlora_i8_linear_fwd(ref(W), X, M, A, B, r, 16.0, ref(drop), Y, U, ws, n, None)
    assert fwd(X=None) == NULL and fwd(Y=None) == NULL and fwd(A=None) == NULL and fwd(M=0) == SHAPE
    assert fwd(M=1 << 40) == SHAPE and fwd(M=(1 << 31) - 1) == UNSUPPORTED and fwd(U=ODD) == ALIGN
    assert fwd(r=0, A=None, B=None, drop=DropDesc(0.1, 1, 1, None)) == UNSUPPORTED
    assert fwd(drop=DropDesc(-0.1, 1, 1, None)) == UNSUPPORTED and fwd(n=100) == WORKSPACE and fwd(ws=None) == NULL

    def bwd(W=rows(), X=P[2], dY=P[3], M=4, A=P[4], B=P[5], r=8, U=None, drop=None, dX=P[6], dA=P[7], dB=P[8], ws=P[9],
            n=1 << 30):
        return L.qlora_i8_linear_bwd(ref(W), X, dY, M, A, B, r, 16.0, U, ref(drop), dX, dA, dB, ws, n, None)
    assert bwd(dY=None) == NULL and bwd(X=None) == NULL and bwd(dA=None) == NULL and bwd(n=100) == WORKSPACE
    assert bwd(r=0, A=None, B=None) == SHAPE      # gradients asked of no adapter
    assert bwd(r=0, A=None, B=None, dA=None, dB=None, drop=DropDesc(0.1, 1, 1, None)) == UNSUPPORTED


def test_adapters_past_32_bit_offsets(L):
    """M r or N r of 2^31 where M K, N K and M N are below it."""
    d = DropDesc(0.1, 1, 2, None)
    for m, n, want in ((1 << 24, 8, UNSUPPORTED), ((1 << 24) - 1, 8, WORKSPACE), (8, 1 << 24, UNSUPPORTED)):
        w = Nf4WeightDesc(n, 64, 64, 256, P[0].value, P[1].value, P[2].value, 0, 0)
        assert L.qlora_linear_fwd_drop(ref(w), P[3], m, P[4], P[5], 128, 16.0, ref(d), P[6], None, P[7], 0, None) == want
        assert L.qlora_linear_bwd_drop(ref(w), P[3], P[8], m, P[4], P[5], 128, 16.0, None, ref(d), P[6], P[9], P[10],
                                       P[7], 0, None) == want
