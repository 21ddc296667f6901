"""GPU: rows of 8-bit integers, their product and the 8-bit linear with its
adapter.  Tolerances are the bounds of tests/test_gpu_dropout.py; codes and
scales are exact."""

import numpy as np
import pytest
import torch

import oracle
from bit_quantized_finetuning_nf4_amd import _lib, ops, synth
from oracle import dropout as OD
from oracle import i8 as OI
from tests.helpers import bits_to_torch, torch_to_bits, torch_to_f64
from tests.test_gpu_dropout import E, F, adapter_bounds, bf16, within

pytestmark = pytest.mark.gpu


def f64(bits):
    return oracle.bf16_bits_to_f64(bits).reshape(bits.shape)


def check_rows(q, x):
    codes, scale = OI.i8_quantize(x)
    got = q.codes.cpu().numpy()
    assert np.array_equal(got[:, :x.shape[1]], codes)
    assert (got[:, x.shape[1]:] == 0).all()
    assert np.array_equal(q.scale.cpu().numpy().view(np.uint32)[~np.isnan(scale)],
                          scale.view(np.uint32)[~np.isnan(scale)])
    assert np.array_equal(np.isnan(q.scale.cpu().numpy()), np.isnan(scale))


@pytest.mark.parametrize("M,K", [(1, 8), (3, 120), (5, 128), (9, 136), (2, 1024), (7, 1032), (4, 4096), (3, 4104),
                                 (2, 8192), (2, 11008), (1, 22016), (2, 32768), (2, 32776), (1, 131072), (1000, 64)])
def test_quantize_rows(M, K):
    print(f"[i8 quantize] M{M} K{K}", flush=True)
    bits = synth.to_bf16_bits(np.random.default_rng(M + K).standard_normal((M, K)))
    out = ops.Int8Weight(M, K, torch.full((M, ops.i8_row_bytes(K)), 55, dtype=torch.int8, device="cuda"),
                         torch.full((M,), 9.0, device="cuda"))
    check_rows(ops.i8_quantize(bits_to_torch(bits).view(M, K), out=out), f64(bits))


def test_quantize_ties_extremes_and_poisoned_rows():
    rng = np.random.default_rng(5)
    rows = []
    for amax in (1.0, 127.0, 254.0, 2.0**-133, 9 * 2.0**-133, 2.0**-126, 3.3e38, 1.9921875, 1.5, 0.0):
        r = np.clip(rng.standard_normal(512) * amax / 3, -amax, amax)
        r[0], r[1], r[2] = amax, -amax / 2, amax / 2   # amax / 2: 63.5 steps, a tie
        rows.append(r)
    bits = synth.to_bf16_bits(np.array(rows))
    x = f64(bits).copy()
    check_rows(ops.i8_quantize(bits_to_torch(bits)), x)
    x[1, 7], x[3, 0], x[4, 511] = np.inf, np.nan, -np.inf
    check_rows(ops.i8_quantize(torch.from_numpy(x).to(torch.bfloat16).cuda()), x)


def test_every_quotient_of_two_significands():
    """All 8-bit significands against all, at distances of 0 to 9 binades."""
    a = (np.arange(128, 256) / 128.0)
    x = np.concatenate([a * 2.0**-d for d in range(10)])
    rows = np.stack([np.concatenate([[m * 2.0], x, np.zeros(7)]) for m in a])   # amax at least every x
    rows = rows[:, : rows.shape[1] // 8 * 8]
    check_rows(ops.i8_quantize(torch.from_numpy(rows).to(torch.bfloat16).cuda()), rows)


@pytest.mark.parametrize("N,K", [(8, 8), (64, 128), (72, 200), (1000, 1032)])
def test_dequant(N, K):
    x, xr = bf16(np.random.default_rng(N), (N, K), 0.02)
    codes, scale = OI.i8_quantize(xr)
    want = oracle.f32_to_bf16_bits(codes.astype(np.float32) * scale[:, None]).reshape(N, K)
    assert np.array_equal(torch_to_bits(ops.i8_dequant(ops.i8_quantize(x))), want)


SHAPES = [
    # M, N, K, r
    (1, 8, 8, 0), (1, 64, 128, 8), (1, 1024, 4096, 64), (2, 4104, 1032, 128), (3, 520, 11008, 16), (5, 96, 264, 0),
    (8, 2048, 2048, 64), (13, 72, 200, 24), (16, 1000, 4096, 8), (17, 264, 1160, 32), (31, 4096, 512, 0),
    (32, 256, 8192, 64), (33, 136, 640, 96), (48, 1032, 1088, 16), (64, 4096, 4096, 64), (65, 320, 2056, 128),
    (100, 776, 576, 8), (128, 264, 1024, 0), (200, 4104, 1024, 16), (256, 1024, 1024, 8), (333, 1376, 4096, 16),
    (513, 264, 320, 128), (1100, 1000, 584, 24), (2048, 5120, 256, 64), (4300, 360, 136, 16),
    # one shape at least for each kernel and launch: lines left over in the streaming kernel's batches, its two
    # widths, two token groups in both widths, 64 x 128, 128 x 128, 192 x 128, 256 x 128 and 256 x 192 tiles, whole
    # rounds of 256 x 256 with the rest apart
    (1, 264, 22016, 8), (9, 8200, 1160, 16), (16, 8192, 384, 0), (4, 22016, 136, 16), (20, 8200, 264, 24),
    (30, 4104, 2056, 8), (200, 4104, 1024, 128), (512, 8192, 256, 16), (333, 11008, 136, 40), (1000, 8192, 128, 64),
    (768, 11008, 128, 8), (2048, 11008, 128, 16), (2000, 11000, 264, 64),
]


@pytest.mark.parametrize("M,N,K,r", SHAPES)
def test_linear(M, N, K, r):
    print(f"[i8 linear] M{M} N{N} K{K} r{r}", flush=True)
    rng = np.random.default_rng(M + N + K + r)
    W, Wr = bf16(rng, (N, K), 0.02)
    X, Xr = bf16(rng, (M, K))
    w = ops.i8_quantize(W)
    (wc, ws), (xc, sx) = OI.i8_quantize(Wr), OI.i8_quantize(Xr)
    main = OI.i8_matmul(xc, sx, wc, ws)
    # the scales' product, and its product with the sum (rounded to fp32 first)
    tol = E * np.abs(main) + 3.01 * 2.0**-24 * np.abs(main)
    within(ops.i8_matmul(ops.i8_quantize(X), w), main, 1.01 * tol, "matmul")
    if r == 0:
        within(ops.i8_linear_fwd(w, X), main, 1.01 * tol, "Y")
        return
    A, Ar = bf16(rng, (r, K), 0.1)
    B, Br = bf16(rng, (N, r), 0.1)
    Y, U = ops.i8_linear_fwd(w, X, A, B, 16.0, save_u=True)
    Y2 = ops.i8_linear_fwd(w, X, A, B, 16.0)
    assert torch.equal(Y, Y2)
    s = 16.0 / r
    Ur = Xr @ Ar.T
    u_err = K * F * (np.abs(Xr) @ np.abs(Ar).T)
    within(U, Ur, 1.01 * (E * np.abs(Ur) + 2 * u_err), "U")
    Yr = main + s * (Ur @ Br.T)
    y_tol = (E * np.abs(Yr) + 4 * 2.0**-24 * np.abs(main)
             + s * ((2.01 * E * np.abs(Ur) + 2 * u_err) @ np.abs(Br).T + r * F * (np.abs(Ur) @ np.abs(Br).T)))
    within(Y, Yr, 1.01 * y_tol, "Y")


@pytest.mark.parametrize("M,N,K,r,p", [(1, 8, 8, 8, 0.5), (70, 72, 200, 8, 0.1), (256, 1024, 1024, 16, 0.0),
                                       (300, 1032, 1096, 64, 0.3), (513, 264, 320, 128, 0.05), (64, 256, 512, 0, 0.0),
                                       (1100, 1000, 584, 96, 0.2)])
def test_backward(M, N, K, r, p):
    print(f"[i8 bwd] M{M} N{N} K{K} r{r} p{p}", flush=True)
    rng = np.random.default_rng(M + N + K + r)
    w = ops.i8_quantize(bf16(rng, (N, K), 0.02)[0])
    Wd = torch_to_f64(ops.i8_dequant(w))
    dY, dYr = bf16(rng, (M, N))
    if r == 0:
        dX, dA, dB = ops.i8_linear_bwd(w, None, dY)
        assert dA is None and dB is None
        ref = dYr @ Wd
        within(dX, ref, 1.01 * (E * np.abs(ref) + N * F * (np.abs(dYr) @ np.abs(Wd))), "dX")
        return
    X, Xr = bf16(rng, (M, K))
    A, Ar = bf16(rng, (r, K), 0.1)
    B, Br = bf16(rng, (N, r), 0.1)
    drop = ops.Dropout(p, 31, 7) if p > 0 else None
    D = OD.keep_mask(M * K, p, 31, 7).reshape(M, K) * OD.keep_scale(p)
    U = ops.i8_linear_fwd(w, X, A, B, 16.0, save_u=True, drop=drop)[1]
    got = ops.i8_linear_bwd(w, X, dY, A, B, 16.0, U=U, drop=drop)
    again = ops.i8_linear_bwd(w, X, dY, A, B, 16.0, drop=drop)   # U computed again
    bounds = adapter_bounds(Xr, dYr, Ar, Br, Wd, 16.0 / r, D, torch_to_f64(U))
    for g, h, (ref, tol), name in zip(got, again, bounds, ("dX", "dA", "dB")):
        within(g, ref, tol, name)
        assert torch.equal(g, h)


def test_a_poisoned_token_stays_alone():
    rng = np.random.default_rng(2)
    w = ops.i8_quantize(bf16(rng, (256, 512), 0.02)[0])
    for M in (3, 40, 300):
        X = bf16(rng, (M, 512))[0]
        want = ops.i8_linear_fwd(w, X)
        X[1, 5] = float("inf")
        got = ops.i8_linear_fwd(w, X)
        assert got[1].isnan().all()
        rest = [i for i in range(M) if i != 1]
        assert torch.equal(got[rest], want[rest])
    # a gradient's infinity stays in its row too (N % 64 != 0: padded rows)
    w = ops.i8_quantize(bf16(rng, (72, 512), 0.02)[0])
    dY = bf16(rng, (40, 72))[0]
    want = ops.i8_linear_bwd(w, None, dY)[0]
    dY[7, 0] = float("inf")
    got = ops.i8_linear_bwd(w, None, dY)[0]
    rest = [i for i in range(40) if i != 7]
    assert torch.equal(got[rest], want[rest])


@pytest.mark.parametrize("M,N,K,r", [(40, 72, 512, 16), (300, 256, 1088, 128)])
def test_an_infinite_gradient_gives_infinite_adapter_gradients(M, N, K, r):
    rng = np.random.default_rng(M)
    w = ops.i8_quantize(bf16(rng, (N, K), 0.02)[0])
    # no zeros: an infinity times any of these is an infinity
    away = lambda shape: bf16(rng, shape)[0].sign().add(0.25)
    X, A, B, dY = away((M, K)), away((r, K)), away((N, r)), away((M, N))
    U = away((M, r))
    dY[7, 3] = float("inf")
    dX, dA, dB = ops.i8_linear_bwd(w, X, dY, A, B, 16.0, U=U)
    G, Xr, Ur = torch_to_f64(dY) @ torch_to_f64(B), torch_to_f64(X), torch_to_f64(U)
    inf_a, inf_b = G.T @ Xr, torch_to_f64(dY).T @ Ur
    assert np.isinf(inf_a).all() and np.array_equal(torch_to_f64(dA), inf_a)
    assert np.isinf(inf_b[3]).all() and np.array_equal(torch_to_f64(dB)[3], inf_b[3])
    rest = [i for i in range(N) if i != 3]
    assert dB[rest].isfinite().all() and dX[:7].isfinite().all() and dX[8:].isfinite().all()


def test_outputs_stay_inside_their_buffers_and_zero_tokens():
    rng = np.random.default_rng(3)
    M, N, K, r = 37, 136, 264, 8
    w = ops.i8_quantize(bf16(rng, (N, K), 0.02)[0])
    X = bf16(rng, (M, K))[0]
    X[4] = 0
    A, B = bf16(rng, (r, K))[0], bf16(rng, (N, r))[0]
    A.zero_()
    whole = torch.full((M * N + 512,), 7.0, dtype=torch.bfloat16, device="cuda")
    Y = ops.i8_linear_fwd(w, X, A, B, 16.0, out=whole[:M * N].view(M, N))
    assert (Y[4] == 0).all() and (whole[M * N:] == 7.0).all()


def test_other_stream_graph_and_two_graphs_of_one_workspace():
    rng = np.random.default_rng(4)
    M, N, K, r = 20, 512, 1024, 16
    w = ops.i8_quantize(bf16(rng, (N, K), 0.02)[0])
    X, A, B = bf16(rng, (M, K))[0], bf16(rng, (r, K))[0], bf16(rng, (N, r))[0]
    X2 = bf16(rng, (3, K))[0]
    want, want2 = ops.i8_linear_fwd(w, X, A, B, 16.0), ops.i8_linear_fwd(w, X2, A, B, 16.0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    ws = torch.empty(ops.workspace_bytes(_lib.QLORA_OP_I8_FWD, M, N, K, r), dtype=torch.uint8, device="cuda")
    Y, Y2 = torch.empty_like(want), torch.empty_like(want2)
    with torch.cuda.stream(side):
        got = ops.i8_linear_fwd(w, X, A, B, 16.0, out=Y, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1, stream=side):
        ops.i8_linear_fwd(w, X, A, B, 16.0, out=Y, ws=ws)
    with torch.cuda.graph(g2, stream=side):
        ops.i8_linear_fwd(w, X2, A, B, 16.0, out=Y2, ws=ws)
    for _ in range(4):   # one after the other on one stream: the workspace is theirs in turn
        Y.zero_(), Y2.zero_()
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want) and torch.equal(Y2, want2)
        assert torch.equal(ops.i8_linear_fwd(w, X, A, B, 16.0), want)


def test_a_training_step_and_decode_together():
    """Quantize, forward under dropout, backward, AdamW, then one decoded
    token with the new adapter, against the oracle."""
    rng = np.random.default_rng(6)
    M, N, K, r, alpha, p = 96, 256, 512, 16, 16.0, 0.2
    W, Wr = bf16(rng, (N, K), 0.02)
    X, Xr = bf16(rng, (M, K))
    dY, dYr = bf16(rng, (M, N), 0.01)
    A, Ar = bf16(rng, (r, K), 0.05)
    B, Br = bf16(rng, (N, r), 0.05)
    w = ops.i8_quantize(W)
    drop = ops.Dropout(p, 3, 1)
    Y, U = ops.i8_linear_fwd(w, X, A, B, alpha, save_u=True, drop=drop)
    dX, dA, dB = ops.i8_linear_bwd(w, X, dY, A, B, alpha, U=U, drop=drop)
    state = {}
    for name, param, grad in (("A", A, dA), ("B", B, dB)):
        master = param.float()
        m, v = torch.zeros_like(master), torch.zeros_like(master)
        ops.adamw(master, grad, m, v, lr=1e-3, step=1, p_bf16=param)
        state[name] = master
    x = X[:1].contiguous()
    y = ops.i8_linear_fwd(w, x, A, B, alpha)
    torch.cuda.synchronize()

    D = OD.keep_mask(M * K, p, 3, 1).reshape(M, K) * OD.keep_scale(p)
    Wd = torch_to_f64(ops.i8_dequant(w))
    bounds = adapter_bounds(Xr, dYr, Ar, Br, Wd, alpha / r, D, torch_to_f64(U))
    for g, (ref, tol), name in zip((dX, dA, dB), bounds, ("dX", "dA", "dB")):
        within(g, ref, tol, name)
    # AdamW's first step moves every value by lr against its gradient's sign
    for name, start, g in (("A", Ar, bounds[1]), ("B", Br, bounds[2])):
        ref, tol = g
        sure = np.abs(ref) > 2 * tol + 1e-4
        moved = state[name].cpu().numpy().astype(np.float64) - start
        assert sure.mean() > 0.5 and (np.sign(moved)[sure] == -np.sign(ref)[sure]).all()
    (wc, ws_), (xc, sx) = OI.i8_quantize(Wr), OI.i8_quantize(Xr[:1])
    A2, B2 = torch_to_f64(A), torch_to_f64(B)
    main = OI.i8_matmul(xc, sx, wc, ws_)
    u = Xr[:1] @ A2.T
    ref = main + alpha / r * (u @ B2.T)
    u_err = K * F * (np.abs(Xr[:1]) @ np.abs(A2).T)
    tol = (E * np.abs(ref) + 4 * 2.0**-24 * np.abs(main)
           + alpha / r * ((2.01 * E * np.abs(u) + 2 * u_err) @ np.abs(B2).T + r * F * (np.abs(u) @ np.abs(B2).T)))
    within(y, ref, 1.01 * tol, "decoded token")


def test_refusals():
    rng = np.random.default_rng(8)
    w = ops.i8_quantize(bf16(rng, (64, 64), 0.02)[0])
    X, A, B = bf16(rng, (4, 64))[0], bf16(rng, (8, 64))[0], bf16(rng, (64, 8))[0]
    with pytest.raises(_lib.QloraError):
        ops.i8_quantize(bf16(rng, (4, 12))[0])                     # cols % 8
    with pytest.raises(ValueError):
        ops.i8_linear_fwd(w, X[:, :56].contiguous())               # K of X and W
    with pytest.raises(ValueError):
        ops.i8_linear_fwd(w, X.float())
    with pytest.raises(ValueError):
        ops.i8_linear_fwd(w, X, A, B[:, :4].contiguous(), 16.0)
    with pytest.raises(_lib.QloraError):
        ops.i8_linear_fwd(w, X, drop=ops.Dropout(0.1, 1))          # no adapter to drop
    with pytest.raises(_lib.QloraError):
        ops.i8_linear_fwd(w, X, A, B, 16.0, drop=ops.Dropout(1.0, 1))
    with pytest.raises(_lib.QloraError):
        ops.i8_linear_fwd(w, X, A, B, 16.0, ws=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(_lib.QloraError):
        ops.i8_linear_fwd(ops.i8_quantize(bf16(rng, (60, 64), 0.02)[0]), X)   # rows % 8
    with pytest.raises(_lib.QloraError):
        ops.i8_matmul(ops.i8_quantize(bf16(rng, (4, 128))[0]), w)
    with pytest.raises(ValueError):
        ops.i8_matmul(ops.Int8Weight(4, 64, torch.zeros(4, 64, dtype=torch.int8, device="cuda"),
                                     torch.zeros(4, device="cuda")), w)       # rows not padded to 128
