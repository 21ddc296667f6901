"""GPU: the products of more than 320 tokens, way by way, adapters included.

Gated block and pools take 256-token tiles of 256, 192 or 128 rows of the stack
(16 of gate and 16 of up in turn), or whole rounds of 256-row tiles and a second
launch for the rows after them; where those would leave CUs idle, small tiles or
a split contraction leave sums that the adapters join in a pass of their own.
Which shape takes which is for 256 CUs.
"""

import numpy as np
import pytest
from tests.test_gpu_gated import block, check_bwd, check_fwd
from tests.test_gpu_many import check, spread_ids

pytestmark = pytest.mark.gpu

# tokens x features x K of a gated block: rows in tiles of 256; of 128; 14336 in whole rounds, then tiles of 128;
# 3840, then of 192; 10752, then of 192
GATED = [(2048, 4096, 64), (700, 4104, 128), (2050, 8208, 128), (4100, 3080, 128), (1300, 8200, 64)]
# of one weight: 256; 3840 in whole rounds, then 192; 14336, then 128
ONE = [(2048, 8192, 128), (4100, 6152, 128), (2050, 16400, 64)]


@pytest.mark.parametrize("M,N,K", GATED)
@pytest.mark.parametrize("r,name", [(24, "gelu"), (64, "silu"), (128, "silu")])
def test_gated_forward_in_every_tile(M, N, K, r, name):
    print(f"[gated_fwd tiles] M={M} F={N} K={K} r={r} {name}", flush=True)
    qs, Ws, X, A, B, _ = block(M + N + r, M, N, K, r)
    check_fwd(qs, Ws, X, A, B, 16.0, name, "tiles")


@pytest.mark.parametrize("M,N,K", GATED)
@pytest.mark.parametrize("R,kind,name", [(16, "outside", "silu"), (64, "runs", "gelu"), (40, "random", "silu")])
def test_gated_many_in_every_tile(M, N, K, R, kind, name):
    print(f"[gated many tiles] M={M} F={N} K={K} R={R} {kind} {name}", flush=True)
    check(M, N, K, 6, R, spread_ids(np.random.default_rng(R), M, 6, kind), M + N + R, G=2, name=name)


@pytest.mark.parametrize("M,N,K", ONE)
@pytest.mark.parametrize("R,kind", [(16, "outside"), (64, "runs"), (128, "random")])
def test_many_in_every_tile(M, N, K, R, kind):
    print(f"[many tiles] M={M} N={N} K={K} R={R} {kind}", flush=True)
    check(M, N, K, 6, R, spread_ids(np.random.default_rng(R), M, 6, kind), M + N + R)


# tokens x features x K, rank: dX's columns in tiles of 256; 3840 in whole rounds, then 192; 14336, then 128
@pytest.mark.parametrize("M,N,K,r", [(2048, 136, 8192, 128), (4100, 136, 6208, 24), (2050, 136, 16448, 16)])
def test_backward_in_every_tile(M, N, K, r):
    print(f"[gated_bwd tiles] M={M} F={N} K={K} r={r}", flush=True)
    qs, Ws, X, A, B, rng = block(M + N, M, N, K, r)
    check_bwd(qs, Ws, X, A, B, 16.0, "silu", rng, "tiles")
