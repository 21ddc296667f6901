"""GPU: the products of more than 320 tokens, way by way, adapters included.

Gated block and pools take 256-token tiles of 256, 192 or 128 rows of the stack
(16 of gate and 16 of up in turn), or whole rounds of 256-row tiles and a second
launch for the rows after them; where those would leave CUs idle, small tiles or
a split contraction leave sums that the adapters join in a pass of their own.
Which shape takes which is for 256 CUs.
"""

import numpy as np
import pytest
import torch

import oracle
from bit_quantized_finetuning_nf4_amd import ops
from tests.test_gpu_gated import E, bf16, block, check_bwd, check_fwd, weight, within
from tests.test_gpu_many import check, make_pool, reference, spread_ids

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


# streamed; small tiles; 256-token tiles in splits, and whole
WAYS = [(1, 5, 136, 128), (1, 300, 136, 128), (1, 400, 136, 128), (1, 1030, 4104, 8192), (1, 2000, 4104, 128),
        (2, 5, 136, 128), (2, 300, 136, 128), (2, 400, 136, 128), (2, 1999, 2104, 128)]


@pytest.mark.parametrize("G,M,N,K", WAYS)
def test_slots_stay_apart(G, M, N, K):
    """Slots that no token names are not read; an infinity or a NaN in a slot's A, B or scale reaches that slot's tokens
    and no other's."""
    print(f"[slots apart] G={G} M={M} N={N} K={K}", flush=True)
    rng = np.random.default_rng(9)
    qs = [weight(rng, N, K)[0] for _ in range(G)]
    X = bf16(rng, (M, K), 0.25)[0]
    p, *_ = make_pool(rng, 4, 16, N, K, G, ranks=[16, 16, 16, 16])
    ids = torch.from_numpy(np.where(np.arange(M) % 2 == 0, 1, 3).astype(np.int32)).cuda()
    run = lambda: ops.many_fwd(qs[0], X, p, ids) if G == 1 else ops.gated_many_fwd(qs, X, p, ids)
    want = run()
    assert torch.isfinite(want).all()
    for t in (p.A, p.B, p.scale):
        t[0] = t[2] = float("nan")
    p.rank[0], p.rank[2] = 2**31 - 1, -2**31
    assert torch.equal(run(), want)
    for t in (p.A, p.B, p.scale):
        for bad in (float("inf"), float("-inf"), float("nan")):
            kept = t[3].clone()
            t[3] = bad
            got = run()
            assert torch.equal(got[::2], want[::2]) and not torch.isfinite(got[1::2]).any()
            t[3] = kept
    assert torch.equal(run(), want)


@pytest.mark.parametrize("G,M,N,K", WAYS)
def test_tokens_stay_apart(G, M, N, K):
    """An infinity or a NaN in one token's row reaches its own outputs alone."""
    print(f"[tokens apart] G={G} M={M} N={N} K={K}", flush=True)
    rng = np.random.default_rng(10)
    qs = [weight(rng, N, K)[0] for _ in range(G)]
    X = bf16(rng, (M, K), 0.25)[0]
    p, *_ = make_pool(rng, 3, 16, N, K, G)
    ids = torch.from_numpy((np.arange(M) % 4 - 1).astype(np.int32)).cuda()
    run = lambda x: ops.many_fwd(qs[0], x, p, ids) if G == 1 else ops.gated_many_fwd(qs, x, p, ids)
    want, x = run(X), X.clone()
    x[M // 2, 5], x[M // 2, 70] = float("inf"), float("nan")
    rest = torch.arange(M, device="cuda") != M // 2
    got = run(x)
    assert torch.equal(got[rest], want[rest]) and got[M // 2].isnan().all()


@pytest.mark.parametrize("M,N,K", [(9, 104, 192), (100, 136, 192), (1040, 4104, 192), (2048, 136, 8192)])
def test_gradients_of_a_token_stay_in_its_row(M, N, K):
    """An infinity in a token's dH, or a NaN in its GU, reaches its own row of dX alone."""
    qs, _, X, A, B, rng = block(M, M, N, K, 16)
    dH, GU, U = bf16(rng, (M, N))[0], bf16(rng, (M, 2 * N))[0], bf16(rng, (M, 32))[0]
    want = ops.gated_bwd(qs, X[0], dH, GU, A[0], B[0], 16.0, U=U)[0]
    rest = torch.arange(M, device="cuda") != M // 2
    for t, bad in ((dH, float("inf")), (GU, float("nan"))):
        t = t.clone()
        t[M // 2, 3] = t[M // 2, N - 1] = bad
        got = ops.gated_bwd(qs, X[0], t if bad == float("inf") else dH, GU if bad == float("inf") else t, A[0], B[0], 16.0,
                            U=U)[0]
        assert torch.equal(got[rest], want[rest]) and not torch.isfinite(got[M // 2]).any()


@pytest.mark.parametrize("M,N,K", [(400, 136, 128), (1030, 520, 320)])
def test_captured_call_in_small_tiles(M, N, K):
    rng = np.random.default_rng(7)
    S, R = 4, 16
    qs = [weight(rng, N, K)[0] for _ in range(2)]
    X = bf16(rng, (M, K))[0]
    p, *_ = make_pool(rng, S, R, N, K, ranks=[16, 8, 16, 16])
    p2, *_ = make_pool(rng, S, R, N, K, G=2)
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    run = lambda: (ops.many_fwd(qs[0], X, p, ids), ops.gated_many_fwd(qs, X, p2, ids))
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = run()
    for k in range(5):
        ids.copy_(torch.from_numpy(rng.integers(-1, S + 1, M).astype(np.int32)))
        p.A[k % S, :8] = bf16(rng, (8, K))[0]
        p.scale[k % S] = 0.25 * k
        p.rank[2] = 8 + 8 * (k % 2)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, run()):
            assert torch.equal(a, b)


def test_streams_in_small_tiles():
    made = []
    for M in (330, 400, 1030):
        rng = np.random.default_rng(M)
        qs = [weight(rng, 264, 192)[0] for _ in range(2)]
        X = bf16(rng, (M, 192))[0]
        p, *_ = make_pool(rng, 3, 16, 264, 192)
        p2, *_ = make_pool(rng, 3, 16, 264, 192, G=2)
        ids = torch.from_numpy((np.arange(M) % 4 - 1).astype(np.int32)).cuda()
        made.append(lambda qs=qs, X=X, p=p, p2=p2, ids=ids: (ops.many_fwd(qs[0], X, p, ids),
                                                            ops.gated_many_fwd(qs, X, p2, ids)))
    want = [run() for run in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    got = []
    for _ in range(3):
        for i, run in enumerate(made):
            with torch.cuda.stream(streams[i]):
                got.append((i, run()))
    torch.cuda.synchronize()
    for i, outs in got:
        for a, b in zip(want[i], outs):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M,N,K,S,R", [(7, 136, 192, 6, 24), (300, 72, 128, 6, 64), (400, 136, 128, 6, 16),
                                       (1999, 4208, 64, 6, 40)])
def test_the_oracles_tokens(M, N, K, S, R):
    """Against oracle.many_fwd, ranks and ids outside the pool included; its error is that of the same sums."""
    rng = np.random.default_rng(M)
    q, W = weight(rng, N, K)
    X = bf16(rng, (M, K), 0.3)
    ranks = [R, 8, 3, 0, -5, 200]
    p, A, B, scale = make_pool(rng, S, R, N, K, ranks=ranks)
    ids = spread_ids(rng, M, S, "outside").astype(np.int32)
    want = oracle.many_fwd(W, X[1], A, B, scale, ids, np.array(ranks))
    _, err = reference([W], X[1], A, B, scale, ids)
    within(ops.many_fwd(q, X[0], p, torch.from_numpy(ids).cuda()), want, E * np.abs(want) + 1.01 * err, "many")
