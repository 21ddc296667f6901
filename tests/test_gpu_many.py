"""GPU: adapters of many requests beside one weight, and beside a gated block's
two.  The bounds are those of tests/test_gpu_gated.py, token by token with the
token's own adapter."""

import math

import numpy as np
import pytest
import torch

import oracle
from bit_quantized_finetuning_nf4_amd import _lib, ops
from tests.helpers import torch_to_f64
from tests.test_gpu_gated import E, bf16, gate_tol, layer_error, weight, within

pytestmark = pytest.mark.gpu


def make_pool(rng, S, R, N, K, G=1, ranks=None):
    """(AdapterPool, its A, B, scale in fp64); a slot's ranks past its own are NaN where they must not be read, zeros
    up to a multiple of eight."""
    A, B = bf16(rng, (S, G * R, K), 0.1), bf16(rng, (S, G * N, R), 0.1)
    scale = (rng.random(S) + 0.5).astype(np.float32)
    a, b = A[0], B[0]
    if ranks is not None:
        for s, r in enumerate(ranks):
            r = max(0, min(R, r))
            r8 = min(R, -(-r // 8) * 8)
            for t, v in ((a[s].view(G, R, K), A[1][s].reshape(G, R, K)),):
                t[:, r:r8] = 0
                v[:, r:r8] = 0
                t[:, r8:] = float("nan")
                v[:, r8:] = 0
            b[s, :, r:r8] = 0
            B[1][s][:, r:r8] = 0
            b[s, :, r8:] = float("nan")
            B[1][s][:, r8:] = 0
    p = ops.AdapterPool(a, b, torch.from_numpy(scale).cuda(),
                        None if ranks is None else torch.tensor(ranks, dtype=torch.int32, device="cuda"))
    return p, A[1], B[1], scale.astype(np.float64)


def reference(Ws, X, A, B, scale, ids):
    """(outputs side by side, the errors that they may have before they are rounded)."""
    G, N = len(Ws), Ws[0].shape[0]
    R = B.shape[2]
    out = [X @ W.T for W in Ws]
    err = [np.zeros_like(y) for y in out]
    for a in sorted(set(ids.tolist())):
        at = np.nonzero(ids == a)[0]
        for g in range(G):
            if 0 <= a < A.shape[0]:
                ag, bg = A[a][g * R:(g + 1) * R], B[a][g * N:(g + 1) * N]
                out[g][at] += scale[a] * ((X[at] @ ag.T) @ bg.T)
                err[g][at] = layer_error(Ws[g], X[at], ag, bg, scale[a])
            else:
                err[g][at] = layer_error(Ws[g], X[at], None, None, 0.0)
    return np.concatenate(out, 1), np.concatenate(err, 1)


def check(M, N, K, S, R, ids, seed, ranks=None, G=1, name="silu", **w):
    rng = np.random.default_rng(seed)
    qs, Ws = zip(*[weight(rng, N, K, **w) for _ in range(G)])
    X = bf16(rng, (M, K), 4.0 / math.sqrt(K))
    p, A, B, scale = make_pool(rng, S, R, N, K, G, ranks)
    ids = np.asarray(ids, dtype=np.int32)
    t = torch.from_numpy(ids).cuda()
    ref, err = reference(Ws, X[1], A, B, scale, ids)
    if G == 1:
        got = ops.many_fwd(qs[0], X[0], p, t)
        within(got, ref, E * np.abs(ref) + 1.01 * err, f"many M={M} N={N} K={K} R={R}")
    else:
        got = ops.gated_many_fwd(list(qs), X[0], p, t, act=name)
        want = oracle.act(ref[:, :N], name)[0] * ref[:, N:]
        within(got, want, gate_tol(ref, err, name), f"gated many M={M} F={N} K={K} R={R}")
    return qs, X, p, t, got


def spread_ids(rng, M, S, kind):
    if kind == "runs":       # packed requests
        cuts = np.sort(rng.integers(0, M + 1, 6))
        return np.searchsorted(cuts, np.arange(M), side="right") % S
    if kind == "random":
        return rng.integers(0, S, M)
    if kind == "own":
        return np.arange(M) % S
    if kind == "none":
        return np.full(M, -1)
    return rng.choice([0, S - 1, S, -1, 2**31 - 1, -2**31, S // 2], M)   # some outside the pool


SHAPES = [(1, 8, 64, 1, 8), (1, 520, 1024, 4, 64), (2, 40, 128, 3, 16), (7, 136, 192, 9, 24), (16, 264, 512, 16, 16),
          (17, 72, 320, 5, 128), (32, 96, 256, 40, 8), (33, 520, 64, 7, 64), (65, 64, 448, 12, 40), (130, 200, 256, 3, 32),
          (300, 1032, 576, 20, 16), (1030, 520, 320, 8, 64),
          # tiles of 256 tokens
          (1999, 4208, 256, 5, 24), (2050, 4104, 192, 300, 8), (1024, 8208, 256, 12, 64), (4100, 2056, 128, 2, 128)]


@pytest.mark.parametrize("M,N,K,S,R", SHAPES)
@pytest.mark.parametrize("kind", ["runs", "random", "own", "none", "outside"])
def test_many(M, N, K, S, R, kind):
    print(f"[many] M={M} N={N} K={K} S={S} R={R} {kind}", flush=True)
    check(M, N, K, S, R, spread_ids(np.random.default_rng(M), M, S, kind), M + N)


@pytest.mark.parametrize("M,N,K,S,R", [s for s in SHAPES if s[0] in (1, 7, 32, 65, 300, 1030)] +
                         [(1999, 2104, 256, 5, 24), (2050, 2056, 192, 300, 8), (1024, 4104, 256, 12, 64), (2300, 2184, 64, 3, 128)])
@pytest.mark.parametrize("kind", ["runs", "outside"])
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_gated_many(M, N, K, S, R, kind, name):
    print(f"[gated many] M={M} F={N} K={K} S={S} R={R} {kind} {name}", flush=True)
    check(M, N, K, S, R, spread_ids(np.random.default_rng(M), M, S, kind), M * N, G=2, name=name)


@pytest.mark.parametrize("M", [1, 9, 40, 200, 1030])
@pytest.mark.parametrize("G", [1, 2])
def test_ranks_of_their_own(M, G):
    """Ranks below R, not multiples of eight, zero, negative and above R; what is past them is NaN and not read."""
    ranks = [64, 8, 3, 0, 40, -5, 17, 200]
    rng = np.random.default_rng(M)
    check(M, 136, 192, 8, 64, rng.integers(0, 8, M), 3, ranks, G)
    check(M, 136, 192, 8, 64, np.sort(rng.integers(0, 8, M)), 4, ranks, G)


@pytest.mark.parametrize("G", [1, 2])
def test_ranks_of_their_own_in_large_tiles(G):
    ranks = [64, 8, 3, 0, 40, -5, 17, 200]
    rng = np.random.default_rng(G)
    check(1999, 4208 // G // 8 * 8, 128, 8, 64, rng.integers(0, 8, 1999), 5, ranks, G)
    check(1999, 4208 // G // 8 * 8, 128, 8, 64, np.sort(rng.integers(-1, 9, 1999)), 6, ranks, G)


@pytest.mark.parametrize("M", [3, 70])
@pytest.mark.parametrize("codebook,fmt", [("fp4", "linear"), ("int4", "fp8"), ("nf4", "fp8")])
def test_codebooks(M, codebook, fmt):
    check(M, 72, 320, 3, 16, np.arange(M) % 3, 5, codebook=codebook, absmax_format=fmt)


@pytest.mark.parametrize("M,N", [(5, 136), (300, 136), (2000, 4104)])
def test_what_no_token_names_is_not_read(M, N):
    rng = np.random.default_rng(9)
    q, _ = weight(rng, N, 128)
    X = bf16(rng, (M, 128))[0]
    p, *_ = make_pool(rng, 4, 16, N, 128)
    ids = torch.from_numpy(np.where(np.arange(M) % 2 == 0, 1, 3).astype(np.int32)).cuda()
    want = ops.many_fwd(q, X, p, ids)
    for t in (p.A, p.B, p.scale):
        t[0] = t[2] = float("nan")
    assert torch.equal(ops.many_fwd(q, X, p, ids), want)
    # an infinity in one slot reaches the tokens of that slot alone
    p.B[3] = float("inf")
    got = ops.many_fwd(q, X, p, ids)
    assert torch.equal(got[::2], want[::2]) and not torch.isfinite(got[1::2]).any()


@pytest.mark.parametrize("M", [1, 3, 40])
def test_token_alone_is_the_linear_layer(M):
    """A pool of one slot against linear_fwd, both within their bounds of the same value."""
    rng = np.random.default_rng(4)
    N, K, r = 264, 256, 16
    q, Wd = weight(rng, N, K)
    X, A, B = bf16(rng, (M, K)), bf16(rng, (r, K), 0.1), bf16(rng, (N, r), 0.1)
    p = ops.AdapterPool(A[0].view(1, r, K), B[0].view(1, N, r), torch.ones(1, device="cuda"))
    got = torch_to_f64(ops.many_fwd(q, X[0], p, torch.zeros(M, dtype=torch.int32, device="cuda")))
    one = torch_to_f64(ops.linear_fwd(q, X[0], A[0], B[0], float(r)))
    assert np.linalg.norm(got - one) <= 1.5 * E * np.linalg.norm(one)


def test_neighbours_and_workspace():
    M, N, K, S, R = 21, 72, 192, 3, 24
    rng = np.random.default_rng(6)
    q, _ = weight(rng, N, K)
    X = bf16(rng, (M, K))[0]
    p, *_ = make_pool(rng, S, R, N, K)
    ids = torch.from_numpy((np.arange(M) % 5 - 1).astype(np.int32)).cuda()
    got = []
    for fill in (0, 255):
        whole = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
        ws = torch.full((ops.workspace_bytes(_lib.QLORA_OP_MANY_FWD, M, N, K, R),), fill, dtype=torch.uint8, device="cuda")
        got.append(ops.many_fwd(q, X, p, ids, out=whole[:M * N].view(M, N), ws=ws))
        assert (whole[M * N:] == 7.0).all()
    assert torch.equal(*got) and torch.isfinite(got[0].float()).all()


@pytest.mark.parametrize("M,N", [(2, 136), (33, 136), (300, 136), (2000, 4104)])
def test_captured_call_follows_ids_and_slots(M, N):
    rng = np.random.default_rng(7)
    K, S, R = 128, 4, 16
    q, _ = weight(rng, N, K)
    qs = [weight(rng, N, K)[0] for _ in range(2)]
    X = bf16(rng, (M, K))[0]
    p, *_ = make_pool(rng, S, R, N, K, ranks=[16, 8, 16, 16])
    p2, *_ = make_pool(rng, S, R, N, K, G=2)
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    run = lambda: (ops.many_fwd(q, X, p, ids), ops.gated_many_fwd(qs, X, p2, ids))
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


def test_refusals():
    rng = np.random.default_rng(8)
    q, _ = weight(rng, 64, 128)
    X = bf16(rng, (4, 128))[0]
    p, *_ = make_pool(rng, 3, 16, 64, 128)
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="ids must be torch.int32"):
        ops.many_fwd(q, X, p, ids.long())
    with pytest.raises(ValueError, match="ids has shape"):
        ops.many_fwd(q, X, p, ids[:3])
    with pytest.raises(ValueError, match="A has shape"):
        ops.gated_many_fwd([q, q], X, p, ids)
    with pytest.raises(ValueError, match="scale has shape"):
        ops.many_fwd(q, X, ops.AdapterPool(p.A, p.B, p.scale[:2]), ids)
    with pytest.raises(ValueError, match="contiguous"):
        ops.many_fwd(q, X, ops.AdapterPool(p.A, p.B.transpose(0, 1).contiguous().transpose(0, 1), p.scale), ids)
    with pytest.raises(ValueError, match="three dimensions"):
        ops.many_fwd(q, X, ops.AdapterPool(p.A[0], p.B[0], p.scale), ids)
    wide = ops.AdapterPool(p.A, torch.zeros(3, 72, 16, dtype=torch.bfloat16, device="cuda"), p.scale)
    with pytest.raises(_lib.QloraError, match="SHAPE"):
        ops.many_fwd(q, X, wide, ids)


def test_feed_forward_block_of_a_serving_batch():
    """Gate and up, activation and down of one batch, each of its requests with its own adapters: a step of decode and
    a packed prompt, the second product on what the first one gave."""
    N, K, S, R = 264, 192, 6, 16
    rng = np.random.default_rng(10)
    qs, Ws = zip(*[weight(rng, N, K) for _ in range(2)])
    down, Wd = weight(rng, K, N // 64 * 64)
    gate_pool, A, B, scale = make_pool(rng, S, R, N, K, G=2)
    down_pool, Ad, Bd, sd = make_pool(rng, S, R, K, N // 64 * 64)
    for M, ids in ((8, np.array([0, 5, -1, 3, 3, 2, 1, 0])), (150, np.repeat([4, 0, 2], 50))):
        ids = ids.astype(np.int32)
        t = torch.from_numpy(ids).cuda()
        X = bf16(rng, (M, K), 0.3)
        H = ops.gated_many_fwd(list(qs), X[0], gate_pool, t)[:, :N // 64 * 64].contiguous()
        ref, err = reference(Ws, X[1], A, B, scale, ids)
        want = oracle.act(ref[:, :N], "silu")[0] * ref[:, N:]
        within(H, want[:, :H.shape[1]], gate_tol(ref, err, "silu")[:, :H.shape[1]], "block H")
        Y = ops.many_fwd(down, H, down_pool, t)
        ref, err = reference([Wd], torch_to_f64(H), Ad, Bd, sd, ids)
        within(Y, ref, E * np.abs(ref) + 1.01 * err, "block Y")
