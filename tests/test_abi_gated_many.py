"""Host-side tests of the gated block's and the adapter pools' entry points
(CPU only: every call here is refused before anything is launched; the pointers
are never read)."""

import ctypes

import pytest
import torch

from bit_quantized_finetuning_nf4_amd import _lib, ops
from bit_quantized_finetuning_nf4_amd._lib import AdapterPoolDesc, Nf4WeightDesc

NULL, ALIGN, SHAPE, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5
P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(12)]
ODD = ctypes.c_void_p(0x10008)
ODD4 = ctypes.c_void_p(0x10002)
BIG = 1 << 60


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def weight(rows=128, cols=256, codes=P[0].value, codebook=0):
    return Nf4WeightDesc(rows, cols, 64, 256, codes, P[1].value, P[2].value, codebook, 0)


def pair(a=None, b=None):
    return (Nf4WeightDesc * 2)(a or weight(), b or weight())


def pool(slots=4, rows=128, cols=256, rank=16, A=P[3].value, B=P[4].value, scale=P[5].value, ranks=None):
    return AdapterPoolDesc(slots, rows, cols, rank, A, B, scale, ranks)


def many(L, W=None, X=P[6], M=4, p=None, ids=P[7], Y=P[8], ws=P[9], n=BIG):
    return L.qlora_many_fwd(ctypes.byref(W or weight()), X, M, ctypes.byref(p or pool()), ids, Y, ws, n, None)


def gated_many(L, W=None, X=P[6], M=4, p=None, ids=P[7], act=0, H=P[8], ws=P[9], n=BIG):
    return L.qlora_gated_many_fwd(W or pair(), X, M, ctypes.byref(p or pool(rows=256)), ids, act, H, ws, n, None)


def gated(L, W=None, X=P[6], M=4, A=P[3], B=P[4], r=16, act=0, H=P[8], GU=None, U=None, ws=P[9], n=BIG):
    return L.qlora_gated_fwd(W or pair(), X, M, A, B, r, 16.0, act, H, GU, U, ws, n, None)


def gated_bwd(L, W=None, X=P[6], dH=P[7], GU=P[8], M=4, A=P[3], B=P[4], r=16, act=0, U=None, dX=P[5], dA=P[10], dB=P[11],
              ws=P[9], n=BIG):
    return L.qlora_gated_bwd(W or pair(), X, dH, GU, M, A, B, r, 16.0, act, U, dX, dA, dB, ws, n, None)


@pytest.mark.parametrize("f", [many, gated_many])
def test_pool(L, f):
    rows = 128 if f is many else 256
    assert f(L, X=None) == NULL and f(L, ids=None) == NULL and f(L, ws=None) == NULL
    assert f(L, X=ODD) == ALIGN and f(L, ids=ODD4) == ALIGN and f(L, ws=ODD) == ALIGN
    assert f(L, M=0) == SHAPE and f(L, M=-1) == SHAPE and f(L, M=1 << 31) == SHAPE
    assert f(L, M=(1 << 31) // 256) == UNSUPPORTED and f(L, n=16) == WORKSPACE
    for k in ("A", "B", "scale"):
        assert f(L, p=pool(rows=rows, **{k: None})) == NULL
    assert f(L, p=pool(rows=rows, A=ODD.value)) == ALIGN and f(L, p=pool(rows=rows, B=ODD.value)) == ALIGN
    assert f(L, p=pool(rows=rows, scale=ODD4.value)) == ALIGN and f(L, p=pool(rows=rows, ranks=ODD4.value)) == ALIGN
    assert f(L, p=pool(rows=rows, slots=0)) == SHAPE and f(L, p=pool(rows=rows + 8)) == SHAPE
    assert f(L, p=pool(rows=rows, cols=320)) == SHAPE and f(L, p=pool(rows=rows, slots=65537)) == UNSUPPORTED
    for rank in (0, -8, 4, 12, 136):
        assert f(L, p=pool(rows=rows, rank=rank)) == UNSUPPORTED


def test_pool_beside_the_wrong_weight(L):
    assert many(L, p=pool(rows=256)) == SHAPE and gated_many(L, p=pool(rows=128)) == SHAPE
    assert many(L, Y=None) == NULL and many(L, Y=ODD) == ALIGN
    assert gated_many(L, H=None) == NULL and gated_many(L, H=ODD) == ALIGN
    assert gated_many(L, act=2) == UNSUPPORTED and gated_many(L, act=-1) == UNSUPPORTED
    assert many(L, W=weight(132)) == UNSUPPORTED and many(L, W=weight(cols=200)) == UNSUPPORTED
    assert gated_many(L, W=pair(weight(), weight(136))) == SHAPE


def test_gated(L):
    for f in (gated, gated_bwd):
        assert f(L, W=pair(weight(), weight(136))) == SHAPE and f(L, W=pair(weight(codes=None))) == NULL
        assert f(L, W=pair(weight(), weight(codebook=3))) == UNSUPPORTED
        assert f(L, W=pair(weight(132), weight(132))) == UNSUPPORTED
        assert f(L, A=None) == NULL and f(L, B=ODD) == ALIGN and f(L, r=12) == UNSUPPORTED and f(L, r=136) == UNSUPPORTED
        assert f(L, M=0) == SHAPE and f(L, M=(1 << 31) // 256) == UNSUPPORTED and f(L, act=2) == UNSUPPORTED
        assert f(L, X=None) == NULL and f(L, X=ODD) == ALIGN and f(L, U=ODD) == ALIGN and f(L, GU=ODD) == ALIGN
        assert f(L, n=16) == WORKSPACE and f(L, ws=None) == NULL and f(L, ws=ODD) == ALIGN
    assert gated(L, H=None) == NULL and gated(L, H=ODD) == ALIGN
    assert gated_bwd(L, dH=None) == NULL and gated_bwd(L, GU=None) == NULL and gated_bwd(L, dH=ODD) == ALIGN
    assert gated_bwd(L, dX=ODD) == ALIGN and gated_bwd(L, dA=None) == NULL and gated_bwd(L, dB=ODD) == ALIGN
    assert gated_bwd(L, r=0, A=None, B=None) == SHAPE
    # nothing asked for: no workspace, nothing launched
    assert gated_bwd(L, r=0, A=None, B=None, dA=None, dB=None, dX=None, X=None, ws=None, n=0) == 0


def test_workspace_is_what_is_asked_for(L):
    for op, f, args in ((_lib.QLORA_OP_GATED_FWD, gated, (4, 128, 256, 16)),
                        (_lib.QLORA_OP_GATED_BWD, gated_bwd, (4, 128, 256, 16)),
                        (_lib.QLORA_OP_MANY_FWD, many, (4, 128, 256, 16)),
                        (_lib.QLORA_OP_GATED_MANY_FWD, gated_many, (4, 128, 256, 16))):
        need = L.qlora_workspace_bytes(op, *args, 0)
        assert need > 0 and f(L, n=need - 1) == WORKSPACE
        for bad in ((0, 128, 256, 16), (4, 0, 256, 16), (4, 128, 0, 16), (4, 128, 200, 16), (4, 128, 256, -8),
                    (4, 128, 256, 256), (1 << 40, 128, 256, 16), (4, 1 << 40, 256, 16), (4, 128, 1 << 40, 16)):
            assert L.qlora_workspace_bytes(op, *bad, 0) == 0, (op, bad)


def test_binding_refuses_before_the_gpu():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    q = ops.QuantizedWeight(8, 64, x, x, x)
    p = ops.AdapterPool(torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(2, 8, 8, dtype=torch.bfloat16),
                        torch.ones(2))
    ids = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: ops.gated_fwd([q, q], x), lambda: ops.gated_bwd([q, q], x, x, x),
                 lambda: ops.many_fwd(q, x, p, ids), lambda: ops.gated_many_fwd([q, q], x, p, ids)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(ValueError, match="activation"):
        ops._act("relu")
