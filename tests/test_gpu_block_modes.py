"""GPU: the gated block and the adapters of many requests where the way a call
is made matters: the debug mode's guards, the numbers of tokens at which the
kernels change, several captured graphs and streams at once, offsets past 32
bits, views at odd places."""

import math

import numpy as np
import pytest
import torch

from bit_quantized_finetuning_nf4_amd import _lib, debug, ops
from tests.helpers import torch_to_f64
from tests.test_gpu_gated import E, F, bf16, block, check_bwd, check_fwd, weight
from tests.test_gpu_many import check, make_pool, spread_ids

pytestmark = pytest.mark.gpu


def bits(t):
    return t.contiguous().view(torch.uint8)


def every_call(M, N=264, K=192, r=16, S=3):
    """Results of each entry point on the same inputs."""
    qs, _, X, A, B, rng = block(M, M, N, K, r)
    p, *_ = make_pool(rng, S, r, N, K)
    p2, *_ = make_pool(rng, S, r, N, K, G=2)
    ids = torch.from_numpy((np.arange(M) % (S + 1) - 1).astype(np.int32)).cuda()
    dH = bf16(rng, (M, N))[0]

    def run():
        H, GU, U = ops.gated_fwd(qs, X[0], A[0], B[0], 16.0, save=True)
        grads = ops.gated_bwd(qs, X[0], dH, GU, A[0], B[0], 16.0, U=U)
        return [H, GU, U, *grads, ops.many_fwd(qs[0], X[0], p, ids), ops.gated_many_fwd(qs, X[0], p2, ids, act="gelu")]
    return run, X[0], ids


@pytest.mark.parametrize("M,N", [(3, 264), (70, 264), (1030, 1032)])
def test_debug_mode(monkeypatch, M, N):
    run, *_ = every_call(M, N)
    plain = run()
    torch.cuda.synchronize()
    monkeypatch.setattr(debug, "ENABLED", True)
    monkeypatch.setattr(debug, "_live", [])
    guarded = run()
    debug.after_call("final check")
    assert all(hasattr(t, "_qlora_guard") and debug.guards_intact(t) for t in guarded)
    for a, b in zip(plain, guarded):
        assert torch.equal(bits(a), bits(b))


# 16 and 32 tokens end a kernel of the streamed product, 64 and 128 a block of it, 320 the streaming
@pytest.mark.parametrize("M", [15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 319, 320, 321, 384])
def test_where_the_kernels_change(M):
    qs, Ws, X, A, B, rng = block(M, M, 264, 320, 24)
    # two codebooks and two formats side by side
    qs[1], Ws[1] = weight(rng, 264, 320, "int4", "fp8")
    check_fwd(qs, Ws, X, A, B, 16.0, "silu", f"M={M}")
    check_bwd(qs, Ws, X, A, B, 16.0, "gelu", rng, f"M={M}")
    check(M, 264, 320, 5, 24, spread_ids(rng, M, 5, "outside"), M)
    check(M, 264, 320, 5, 24, spread_ids(rng, M, 5, "runs"), M, G=2)


def test_repeated_calls_agree_bit_for_bit():
    for M in (1, 33, 64, 200, 1030):
        run, *_ = every_call(M, 1032)
        first = run()
        for _ in range(3):
            for a, b in zip(first, run()):
                assert torch.equal(bits(a), bits(b))


def test_two_graphs_in_turn():
    """Two captured graphs, each with workspaces of its own, replayed in turn with eager calls between."""
    made = []
    for M in (5, 130):
        run, X, ids = every_call(M)
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = run()
        made.append((g, outs, run, X, ids))
    for k in range(4):
        for g, outs, run, X, ids in made:
            X.mul_(0.75)
            ids.copy_(ids.roll(1))
            g.replay()
        torch.cuda.synchronize()
        for g, outs, run, X, ids in made:
            for a, b in zip(outs, run()):
                assert torch.equal(bits(a), bits(b)), k


def test_streams_of_their_own():
    runs = [every_call(M)[0] for M in (4, 66, 300)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = []
    for _ in range(3):
        for i, run in enumerate(runs):
            with torch.cuda.stream(streams[i]):
                got.append((i, run()))
    torch.cuda.synchronize()
    for i, outs in got:
        for a, b in zip(want[i], outs):
            assert torch.equal(bits(a), bits(b))


def test_views_inside_larger_tensors():
    """Tokens that are rows of a longer batch, slots that are part of a larger pool; odd places are refused."""
    rng = np.random.default_rng(2)
    N, K, R = 136, 192, 16
    q, _ = weight(rng, N, K)
    X = bf16(rng, (40, K))[0]
    p, *_ = make_pool(rng, 6, R, N, K)
    ids = torch.from_numpy((np.arange(40) % 3).astype(np.int32)).cuda()
    part = ops.AdapterPool(p.A[2:5], p.B[2:5], p.scale[2:5])
    got = ops.many_fwd(q, X[7:20], part, ids[7:20])
    whole = ops.many_fwd(q, X[7:20].clone(), p, ids[7:20] + 2)
    assert torch.equal(got, whole)
    room = torch.zeros(13 * N + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(_lib.QloraError, match="ALIGN"):
        ops.many_fwd(q, X[7:20], part, ids[7:20], out=room[1:1 + 13 * N].view(13, N))
    with pytest.raises(ValueError, match="contiguous"):
        ops.many_fwd(q, X[::2], part, ids[:20])
    with pytest.raises(ValueError, match="contiguous"):
        ops.many_fwd(q, X[:20], part, ids[::2])


def test_no_tokens_is_refused():
    rng = np.random.default_rng(3)
    q, _ = weight(rng, 64, 128)
    p, *_ = make_pool(rng, 2, 8, 64, 128)
    none = torch.zeros(0, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(_lib.QloraError, match="SHAPE"):
        ops.many_fwd(q, none, p, torch.zeros(0, dtype=torch.int32, device="cuda"))
    with pytest.raises(_lib.QloraError, match="SHAPE"):
        ops.gated_fwd([q, q], none)


def test_a_token_of_infinities_stays_alone():
    """An infinity or a NaN in one token's row reaches that token's outputs and no other's."""
    for M in (9, 100, 1030):
        qs, _, X, A, B, rng = block(M, M, 1032, 192, 16)
        p, *_ = make_pool(rng, 3, 16, 1032, 192)
        ids = torch.from_numpy((np.arange(M) % 3).astype(np.int32)).cuda()
        x = X[0].clone()
        x[M // 2, 5], x[M // 2, 70] = float("inf"), float("nan")
        rest = torch.arange(M, device="cuda") != M // 2
        for f in (lambda v: ops.gated_fwd(qs, v, A[0], B[0], 16.0), lambda v: ops.many_fwd(qs[0], v, p, ids)):
            want, got = f(X[0]), f(x)
            assert torch.equal(got[rest], want[rest]) and got[M // 2].isnan().all()


def big_weight(N, K):
    """Random codes made on the GPU; (QuantizedWeight, one of its last rows alone)."""
    blocks = N * K // 64
    codes = torch.randint(0, 256, (N * K // 2,), dtype=torch.uint8, device="cuda")
    aq = torch.randint(0, 256, (blocks,), dtype=torch.uint8, device="cuda")
    s2 = torch.rand(blocks // 256, device="cuda") * 0.1 + 0.1
    return ops.QuantizedWeight(N, K, codes, aq, s2)


def rows_of(q, at, n):
    """Rows at .. at + n of q as a weight of its own (K a multiple of 64 x 256)."""
    K = q.cols
    return ops.QuantizedWeight(n, K, q.codes[at * K // 2:(at + n) * K // 2].clone(),
                               q.absmax_q[at * K // 64:(at + n) * K // 64].clone(),
                               q.group_scale[at * K // 16384:(at + n) * K // 16384].clone())


@pytest.mark.parametrize("M", [2, 40, 80, 330])
def test_a_weight_of_two_to_the_31(M):
    """The last rows of 2^31 - 2^17 weights, whose byte offsets do not fit 31 bits (2^32 as bf16), are those of the rows
    alone.  Both sides are off by their sum and their rounding."""
    N, K, R, S = 131064, 16384, 8, 2
    torch.manual_seed(0)
    rng = np.random.default_rng(0)
    q = big_weight(N, K)
    X = bf16(rng, (M, K), 4.0 / math.sqrt(K))[0]
    A = bf16(rng, (S, R, K), 0.1)[0]
    B = torch.randn(S, N, R, device="cuda").to(torch.bfloat16)
    scale = torch.ones(S, device="cuda")
    ids = torch.from_numpy((np.arange(M) % S).astype(np.int32)).cuda()
    Y = ops.many_fwd(q, X, ops.AdapterPool(A, B, scale), ids)
    for at in (0, N // 2, N - 8):
        one = rows_of(q, at, 8)
        W = ops.dequant(one).view(8, K).double()
        T = X.double() @ A.double().transpose(1, 2)   # [S, M, R]
        part = B[:, at:at + 8].double()
        want = X.double() @ W.T
        size = X.double().abs() @ W.abs().T
        for s in range(S):
            mine = ids == s
            want[mine] += T[s][mine] @ part[s].T
            size[mine] += (X.double().abs() @ A[s].double().abs().T)[mine] @ part[s].abs().T
        tol = E * want.abs() + 1.01 * (K + R) * F * size
        assert ((Y[:, at:at + 8].double() - want).abs() <= tol).all(), at
    # two of half the rows make a block of as many
    half = 65504   # whole 32s, as the block's stack is laid out
    qs = [rows_of(q, 0, half), rows_of(q, half, half)]
    H, GU, _ = ops.gated_fwd(qs, X, save=True)
    for g in range(2):
        for at in (0, half - 8):
            W = ops.dequant(rows_of(qs[g], at, 8)).view(8, K).double()
            want, size = X.double() @ W.T, X.double().abs() @ W.abs().T
            got = GU[:, g * half + at:g * half + at + 8].double()
            assert ((got - want).abs() <= E * want.abs() + 1.01 * K * F * size).all(), (g, at)


def test_tokens_of_two_to_the_31():
    """X of 2^31 - 2^16 elements: the last tokens are what they are alone."""
    M, N, K, R, S = 1048544, 64, 2048, 8, 3
    rng = np.random.default_rng(1)
    q, _ = weight(rng, N, K)
    X = torch.randn(M, K, device="cuda", dtype=torch.bfloat16)
    p, *_ = make_pool(rng, S, R, N, K)
    ids = torch.arange(M, device="cuda", dtype=torch.int32) % S
    Y = ops.many_fwd(q, X, p, ids)
    W = ops.dequant(q).view(N, K).double()
    for at in (0, M // 2, M - 40):
        x = X[at:at + 40].double()
        T = x @ p.A.double().transpose(1, 2) * p.scale.double()[:, None, None]
        want, size = x @ W.T, x.abs() @ W.abs().T
        for s in range(S):
            mine = ids[at:at + 40] == s
            want[mine] += T[s][mine] @ p.B[s].double().T
            size[mine] += (x.abs() @ p.A[s].double().abs().T * p.scale[s].double())[mine] @ p.B[s].double().abs().T
        # T may enter as two bf16 parts, 2^-17 of it
        tol = E * want.abs() + 1.01 * ((K + R) * F + 2.0**-17) * size
        assert ((Y[at:at + 40].double() - want).abs() <= tol).all(), at


# (tokens, features, K, rank): 256-token tiles for dX, whole and in a split contraction
@pytest.mark.parametrize("M,N,K,r", [(2050, 104, 8192, 24), (2050, 200, 4160, 0), (1040, 4104, 4160, 72), (1040, 4104, 4096, 0),
                                     (2050, 4104, 2048, 128)])
def test_backward_in_large_tiles(M, N, K, r):
    print(f"[gated_bwd] M={M} F={N} K={K} r={r}", flush=True)
    qs, Ws, X, A, B, rng = block(M, M, N, K, r)
    check_bwd(qs, Ws, X, A, B, 16.0, "silu", rng, "large tiles")


def test_many_in_a_split_contraction():
    check(1030, 4104, 8192, 6, 40, spread_ids(np.random.default_rng(3), 1030, 6, "outside"), 3)


def test_a_block_of_a_million_features():
    """More rows than a grid's second dimension could count; the first and last 256 are what they are alone."""
    M, N, K = 330, 1200128, 64   # 256 x 4688
    torch.manual_seed(2)
    qs = [big_weight(N, K) for _ in range(2)]
    X = bf16(np.random.default_rng(2), (M, K), 0.5)[0]
    H, GU, _ = ops.gated_fwd(qs, X, save=True)
    for at in (0, N - 256):
        for g, q in enumerate(qs):
            one = ops.QuantizedWeight(256, K, q.codes[at * 32:(at + 256) * 32].clone(), q.absmax_q[at:at + 256].clone(),
                                      q.group_scale[at // 256:at // 256 + 1].clone())
            W = ops.dequant(one).view(256, K).double()
            want, size = X.double() @ W.T, X.double().abs() @ W.abs().T
            got = GU[:, g * N + at:g * N + at + 256].double()
            assert ((got - want).abs() <= E * want.abs() + 1.01 * K * F * size).all(), (g, at)
    assert torch.isfinite(H).all()


@pytest.mark.parametrize("K", [64, 128, 192, 320, 448, 576, 1088, 1216])
@pytest.mark.parametrize("N", [8, 24, 32, 40, 104, 264])
def test_rows_whose_block_codes_share_words(N, K):
    """K / 64 of 1 to 19 block codes a row, at every place in a word, the array ending inside one or not."""
    for M in (1, 20, 40):
        check(M, N, K, 3, 8, np.arange(M) % 4 - 1, M + N + K)
