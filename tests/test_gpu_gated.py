"""GPU: the gated feed-forward block, forward and backward.

Tolerances are bounds, element by element.  bf16 rounds by at most E = 2^-8 of
the value, fp32 by 2^-24; a sum of n fp32 products in any order is off by at
most n 2^-23 = n F of the sum of their magnitudes (n additions and n products,
2^-24 each).  s U enters a product in fp32, or as two bf16 parts (2^-17 of it).
act has slopes up to 1.2 and is itself off by at most (2 |p| + 8) 2^-22 of its
value, |p| its exponent's argument (the argument's rounding and the hardware's
exponential).
"""

import math

import numpy as np
import pytest
import torch

import oracle
from bit_quantized_finetuning_nf4_amd import ops, synth
from tests.helpers import bits_to_torch, torch_to_bits, torch_to_f64

pytestmark = pytest.mark.gpu

E = 2.0**-8
F = 2.0**-23


def bf16(rng, shape, std=1.0):
    """(GPU tensor, its values in fp64)."""
    bits = synth.to_bf16_bits(rng.standard_normal(shape) * std)
    return bits_to_torch(bits), oracle.bf16_bits_to_f64(bits).reshape(shape)


def weight(rng, N, K, codebook="nf4", absmax_format="linear", scale=0.1):
    """(QuantizedWeight of random codes, deq(W) in fp64)."""
    blocks = -(-N * K // 64)
    codes = rng.integers(0, 256, -(-N * K // 2), dtype=np.uint8)
    if codebook == "fp4":   # code 8 is never produced
        codes = np.where((codes & 15) == 8, codes - 1, codes)
        codes = np.where((codes >> 4) == 8, codes - 16, codes).astype(np.uint8)
    aq = rng.integers(0, 127 if absmax_format == "fp8" else 256, blocks, dtype=np.uint8)
    s2 = (rng.random(-(-blocks // 256)) * scale + scale).astype(np.float32)
    t = lambda a: torch.from_numpy(a.copy()).cuda()
    q = ops.QuantizedWeight(N, K, t(codes), t(aq), t(s2), codebook, absmax_format)
    return q, oracle.bf16_bits_to_f64(oracle.dequant(codes, aq, s2, N * K, codebook, absmax_format)).reshape(N, K)


def within(got, ref, tol, name):
    got = torch_to_f64(got)
    assert got.shape == ref.shape and np.isfinite(got).all(), name
    over = np.abs(got - ref) - (tol + 1e-37)
    assert (over <= 0).all(), f"{name}: {over.max():.3e} over its bound, {(over > 0).sum()} of {over.size}"


def layer_error(Wd, X, A, B, s):
    """The error that a layer's fp32 sum may have before it is rounded (A None: no adapter)."""
    K = X.shape[1]
    err = K * F * (np.abs(X) @ np.abs(Wd).T)
    if A is None or A.shape[0] == 0:
        return err + F * np.abs(X @ Wd.T)
    r = A.shape[0]
    T = np.abs(X) @ np.abs(A).T
    U = np.abs(X @ A.T)
    err += s * ((K * F * T + (2.0**-16 + r * F) * U) @ np.abs(B).T)
    return err + 4 * F * (np.abs(X @ Wd.T) + s * (U @ np.abs(B).T))


def gate_tol(GU, err, name):
    """The bound of H from those of G and P."""
    n = GU.shape[1] // 2
    g, p, eg, ep = GU[:, :n], GU[:, n:], err[:, :n], err[:, n:]
    a = oracle.act(g, name)[0]
    arg = np.abs(g) if name == "silu" else 1.6 * np.abs(g + 0.044715 * g**3)
    ea = 1.2 * eg + np.abs(a) * (2 * np.minimum(arg, 100) + 8) * 2.0**-22 + 1e-36
    return E * np.abs(a * p) + 1.01 * (ea * np.abs(p) + np.abs(a) * ep + ea * ep)


def block(seed, M, N, K, r, **w):
    rng = np.random.default_rng(seed)
    qs, Ws = zip(*[weight(rng, N, K, **w) for _ in range(2)])
    X = bf16(rng, (M, K), 4.0 / math.sqrt(K))
    A = bf16(rng, (2 * r, K), 0.1) if r else (None, None)
    B = bf16(rng, (2 * N, r), 0.1) if r else (None, None)
    return list(qs), list(Ws), X, A, B, rng


def check_fwd(qs, Ws, X, A, B, alpha, name, label):
    N = qs[0].rows
    r = 0 if A[1] is None else A[1].shape[0] // 2
    H, GU, U = ops.gated_fwd(qs, X[0], A[0], B[0], alpha, act=name, save=True)
    Href, GUref = oracle.gated_fwd(Ws, X[1], A[1], B[1], alpha, name)
    s = oracle.lora_scale(alpha, r)
    half = lambda t, i: None if t is None else np.split(t, 2)[i]
    err = np.concatenate([layer_error(Ws[i], X[1], half(A[1], i), half(B[1], i), abs(s)) for i in range(2)], axis=1)
    within(GU, GUref, E * np.abs(GUref) + 1.01 * err, f"{label} GU")
    within(H, Href, gate_tol(GUref, err, name), f"{label} H")
    if r:
        Uref = X[1] @ A[1].T
        within(U, Uref, E * np.abs(Uref) + 1.01 * X[1].shape[1] * F * (np.abs(X[1]) @ np.abs(A[1]).T), f"{label} U")
    else:
        assert U is None
    assert torch.equal(H, ops.gated_fwd(qs, X[0], A[0], B[0], alpha, act=name)), f"{label}: H without save"
    return H, GU, U


SHAPES = [(1, 8, 64, 8), (1, 256, 1024, 64), (2, 40, 128, 0), (5, 136, 192, 24), (16, 264, 512, 16), (17, 64, 320, 8),
          (32, 96, 256, 128), (33, 520, 64, 64), (63, 72, 448, 40), (130, 200, 256, 32), (257, 328, 128, 16),
          (300, 1032, 576, 72), (1024, 512, 256, 64), (1030, 2056, 320, 8),
          # tiles of 256 tokens: ragged tokens, features and ranks
          (1999, 2104, 256, 24), (2050, 2056, 192, 128), (1024, 4104, 256, 64), (4100, 1032, 256, 0), (2300, 2184, 128, 8)]


@pytest.mark.parametrize("M,N,K,r", SHAPES)
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_forward(M, N, K, r, name):
    print(f"[gated_fwd] M={M} F={N} K={K} r={r} {name}", flush=True)
    qs, Ws, X, A, B, _ = block(M + N, M, N, K, r)
    check_fwd(qs, Ws, X, A, B, 16.0, name, "forward")


@pytest.mark.parametrize("codebook", ["nf4", "fp4", "int4"])
@pytest.mark.parametrize("fmt", ["linear", "fp8"])
@pytest.mark.parametrize("M", [3, 70])
def test_codebooks(codebook, fmt, M):
    qs, Ws, X, A, B, rng = block(7, M, 72, 320, 16, codebook=codebook, absmax_format=fmt)
    check_fwd(qs, Ws, X, A, B, 16.0, "silu", f"{codebook} {fmt}")
    # the two weights may differ in both
    qs[1], Ws[1] = weight(rng, 72, 320, "int4" if codebook == "nf4" else "nf4", "fp8" if fmt == "linear" else "linear")
    _, GU, U = check_fwd(qs, Ws, X, A, B, 16.0, "silu", "mixed")
    check_bwd(qs, Ws, X, A, B, 16.0, "silu", rng, "mixed")


def check_bwd(qs, Ws, X, A, B, alpha, name, rng, label, give_u=True):
    N, K, M = qs[0].rows, qs[0].cols, X[1].shape[0]
    r = 0 if A[1] is None else A[1].shape[0] // 2
    s = oracle.lora_scale(alpha, r)
    dH, GU = bf16(rng, (M, N)), bf16(rng, (M, 2 * N), 2.0)
    U = bf16(rng, (M, 2 * r)) if r and give_u else (None, None)
    dX, dA, dB = ops.gated_bwd(qs, X[0], dH[0], GU[0], A[0], B[0], alpha, act=name, U=U[0])
    dY = np.split(oracle.gated_dy(dH[1], GU[1], name), 2, axis=1)
    ref, tol = np.zeros((M, K)), np.zeros((M, K))
    for i in range(2):
        ref += dY[i] @ Ws[i]
        tol += 2 * N * F * (np.abs(dY[i]) @ np.abs(Ws[i]))
    for i in range(2 if r else 0):
        a, b = np.split(A[1], 2)[i], np.split(B[1], 2)[i]
        G, Gm = dY[i] @ b, np.abs(dY[i]) @ np.abs(b)
        ref += s * (G @ a)
        # s G in two bf16 parts, 2^-17 of it
        tol += s * ((2.0**-16 * np.abs(G) + (N + 2) * F * Gm) @ np.abs(a) + 2 * r * F * (np.abs(G) @ np.abs(a)))
        # in three (2^-24), then a sum over the tokens
        da = s * (G.T @ X[1])
        da_tol = s * ((2.0**-23 * np.abs(G) + (N + 2) * F * Gm).T @ np.abs(X[1]) + 3 * M * F * (np.abs(G).T @ np.abs(X[1])))
        within(dA[i * r:(i + 1) * r], da, 1.01 * da_tol, f"{label} dA {i}")
        if give_u:
            u, u_tol = U[1][:, i * r:(i + 1) * r], 0.0
        else:   # computed again, in bf16
            u = X[1] @ a.T
            u_tol = 1.01 * (E * np.abs(u) + K * F * (np.abs(X[1]) @ np.abs(a).T))
        db_tol = s * ((M + 2) * F * (np.abs(dY[i]).T @ np.abs(u)) + np.abs(dY[i]).T @ (u_tol + 0 * u))
        within(dB[i * N:(i + 1) * N], s * (dY[i].T @ u), 1.01 * db_tol, f"{label} dB {i}")
    within(dX, ref, 1.01 * (E * np.abs(ref) + tol), f"{label} dX")
    return dH, GU, U, dX, dA, dB


BWD = [(1, 8, 64, 8), (3, 40, 128, 0), (16, 136, 192, 24), (31, 32, 64, 64), (64, 256, 320, 128), (130, 200, 256, 72),
       (257, 520, 128, 16), (300, 1032, 576, 32), (1040, 512, 256, 64)]


@pytest.mark.parametrize("M,N,K,r", BWD)
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_backward(M, N, K, r, name):
    print(f"[gated_bwd] M={M} F={N} K={K} r={r} {name}", flush=True)
    qs, Ws, X, A, B, rng = block(M * N, M, N, K, r)
    check_bwd(qs, Ws, X, A, B, 16.0, name, rng, "backward")


def test_backward_computes_u_again_and_skips_dx():
    qs, Ws, X, A, B, rng = block(3, 70, 104, 192, 16)
    dH, GU, U, dX, dA, dB = check_bwd(qs, Ws, X, A, B, 16.0, "silu", rng, "no U", give_u=False)
    none, dA2, dB2 = ops.gated_bwd(qs, X[0], dH[0], GU[0], A[0], B[0], 16.0, need_dx=False)
    assert none is None and torch.equal(dA, dA2) and torch.equal(dB, dB2)
    dX2, nA, nB = ops.gated_bwd(qs, None, dH[0], GU[0])
    assert nA is None and nB is None
    assert ops.gated_bwd(qs, None, dH[0], GU[0], need_dx=False) == (None, None, None)


def test_gradients_are_differences():
    # the loss sum(dH o H) along one direction of X, A and B; H is rounded, so the step is large and the bound the
    # step's curvature and H's roundings: |H| <= 4, slopes below 1.2, second derivatives below 1
    M, N, K, r, alpha = 48, 64, 128, 16, 16.0
    qs, Ws, X, A, B, rng = block(11, M, N, K, r)
    dH = bf16(rng, (M, N))
    _, GU, U = ops.gated_fwd(qs, X[0], A[0], B[0], alpha, save=True)
    grads = [torch_to_f64(g) for g in ops.gated_bwd(qs, X[0], dH[0], GU, A[0], B[0], alpha, U=U)]
    base = [X[1], A[1], B[1]]
    for i, g in enumerate(grads):
        d = rng.standard_normal(base[i].shape) * np.abs(base[i]).mean() * 0.5
        ends = []
        for sign in (1, -1):
            bits = synth.to_bf16_bits(base[i] + sign * d)
            ends.append((bits_to_torch(bits), oracle.bf16_bits_to_f64(bits).reshape(base[i].shape)))
        H = []
        for t, _ in ends:
            args = [X[0], A[0], B[0]]
            args[i] = t
            H.append(torch_to_f64(ops.gated_fwd(qs, *args, alpha)))
        got = float((dH[1] * (H[0] - H[1])).sum())
        want = float((g * (ends[0][1] - ends[1][1])).sum())
        # the exact loss at the same ends says how much of it the straight line misses
        exact = []
        for _, v in ends:
            args = [base[0], base[1], base[2]]
            args[i] = v
            exact.append(oracle.gated_fwd(Ws, *args, alpha, "silu")[0])
        line = float((dH[1] * (exact[0] - exact[1])).sum())
        rounding = float((np.abs(dH[1]) * E * 1.05 * (np.abs(exact[0]) + np.abs(exact[1]))).sum())
        assert abs(got - line) <= rounding
        # GU, U, dG and dP are rounded by E each (GU moves the slopes by up to E |x| of order 1), dX once more
        slack = 8 * E * float((np.abs(g) * np.abs(ends[0][1] - ends[1][1])).sum()) + abs(line - want_exact(Ws, base, dH[1], alpha, i, ends))
        assert abs(want - line) <= slack


def want_exact(Ws, base, dH, alpha, i, ends):
    GU = oracle.gated_fwd(Ws, *base, alpha, "silu")[1]
    g = oracle.gated_bwd(Ws, base[0], dH, GU, base[1], base[2], alpha, "silu")[i]
    return float((g * (ends[0][1] - ends[1][1])).sum())


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_gate_at_its_ends(name):
    """dG and dP of gates from -inf to inf, infinities and NaN: the oracle's bits, except where both are NaN."""
    g = np.array([0.0, -0.0, 1e-30, -1e-30, 3e38, -3e38, 90.0, -90.0, 750.0, -750.0, 1.2e4, -1.2e4, 1e13, -1e13, np.inf,
                  -np.inf, np.nan, 1.0, -1.0, -0.75, -1.28, -12.0, 12.0, -30.0])
    N, K = len(g), 64
    qs = [weight(np.random.default_rng(0), N, K)[0] for _ in range(2)]
    one = np.ones((1, N))
    to = lambda a: bits_to_torch(synth.to_bf16_bits(np.nan_to_num(a, nan=0.0))) if not np.isnan(a).any() else (
        torch.from_numpy(a).to(torch.bfloat16).cuda())
    GU = to(np.concatenate((g[None], 1.5 * one), axis=1))
    # dX of an identity-like weight is not needed: a single adapter of rank 8 reads dG and dP out through dB
    r = 8
    A = torch.zeros(2 * r, K, dtype=torch.bfloat16, device="cuda")
    B = torch.zeros(2 * N, r, dtype=torch.bfloat16, device="cuda")
    U = torch.zeros(1, 2 * r, dtype=torch.bfloat16, device="cuda")
    U[0, 0] = U[0, r] = 1.0
    X = torch.zeros(1, K, dtype=torch.bfloat16, device="cuda")
    _, _, dB = ops.gated_bwd(qs, X, to(one * 2.0), GU, A, B, float(r), act=name, U=U, need_dx=False)
    got = torch_to_f64(dB)[:, 0]
    with np.errstate(all="ignore"):
        ref = oracle.gated_dy(2.0 * one, torch_to_f64(GU.float()), name)[0]
        assert np.array_equal(np.isfinite(got), np.isfinite(ref))
        ok = np.isfinite(ref)
        assert np.array_equal(got[ok], ref[ok])


def test_neighbours_stay_as_they_were():
    M, N, K, r = 37, 72, 128, 8
    qs, Ws, X, A, B, rng = block(5, M, N, K, r)
    def inside(shape, dtype):
        whole = torch.full((int(np.prod(shape)) + 64,), 7.0, dtype=dtype, device="cuda")
        return whole, whole[:int(np.prod(shape))].view(shape)
    bufs = [inside((M, N), torch.bfloat16), inside((M, 2 * N), torch.bfloat16), inside((M, 2 * r), torch.bfloat16)]
    H, GU, U = ops.gated_fwd(qs, X[0], A[0], B[0], 16.0, save=True, out=bufs[0][1], gu_out=bufs[1][1], u_out=bufs[2][1])
    assert H.data_ptr() == bufs[0][0].data_ptr()
    gb = [inside((M, K), torch.bfloat16), inside((2 * r, K), torch.float32), inside((2 * N, r), torch.float32)]
    ops.gated_bwd(qs, X[0], H, GU, A[0], B[0], 16.0, U=U, dX=gb[0][1], dA=gb[1][1], dB=gb[2][1])
    for whole, view in bufs + gb:
        assert (whole[view.numel():] == 7.0).all()


def test_workspace_contents_do_not_matter():
    from bit_quantized_finetuning_nf4_amd import _lib
    M, N, K, r = 50, 40, 192, 24   # F not a multiple of 32: padded columns
    qs, Ws, X, A, B, rng = block(6, M, N, K, r)
    dH, GU = bf16(rng, (M, N)), bf16(rng, (M, 2 * N))
    got = []
    for fill in (0, 255):   # 255: NaNs
        ws = torch.full((ops.workspace_bytes(_lib.QLORA_OP_GATED_BWD, M, N, K, r),), fill, dtype=torch.uint8, device="cuda")
        bw = ops.gated_bwd(qs, X[0], dH[0], GU[0], A[0], B[0], 16.0, ws=ws)
        ws = torch.full((ops.workspace_bytes(_lib.QLORA_OP_GATED_FWD, M, N, K, r),), fill, dtype=torch.uint8, device="cuda")
        got.append(bw + ops.gated_fwd(qs, X[0], A[0], B[0], 16.0, save=True, ws=ws))
    for a, b in zip(*got):
        assert torch.isfinite(a.float()).all() and torch.equal(a, b)


def test_refusals():
    qs, Ws, X, A, B, rng = block(8, 4, 16, 64, 8)
    with pytest.raises(ValueError, match="two weights"):
        ops.gated_fwd(qs[:1], X[0])
    with pytest.raises(ValueError, match="X has shape"):
        ops.gated_fwd(qs, torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        ops.gated_fwd(qs, torch.zeros(64, 4, dtype=torch.bfloat16, device="cuda").t())
    with pytest.raises(ValueError, match="B has shape"):
        ops.gated_fwd(qs, X[0], A[0], B[0][:16].contiguous(), 16.0)
    with pytest.raises(ValueError, match="activation"):
        ops.gated_fwd(qs, X[0], act="relu")
    with pytest.raises(ValueError, match="GU has shape"):
        ops.gated_bwd(qs, X[0], torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda"), X[0])
    short = ops.QuantizedWeight(16, 64, qs[0].codes[:16], qs[0].absmax_q, qs[0].group_scale)
    with pytest.raises(ValueError, match="codes holds"):
        ops.gated_fwd([short, qs[1]], X[0])


def test_training_pass_of_a_feed_forward_block():
    """Norm-free block: gate and up, activation, down, and back, against the oracle's whole chain (each stage's own
    inputs, so that the bounds stay those of one stage)."""
    M, N, K, r, alpha = 200, 192, 128, 16, 16.0
    qs, Ws, X, A, B, rng = block(12, M, N, K, r)
    down, Wd = weight(rng, K, N)
    Ad, Bd = bf16(rng, (r, N), 0.1), bf16(rng, (K, r), 0.1)
    H, GU, U = check_fwd(qs, Ws, X, A, B, alpha, "silu", "block")
    Y, Ud = ops.linear_fwd(down, H, Ad[0], Bd[0], alpha, save_u=True)
    dY = bf16(rng, (M, K))
    dH, dAd, dBd = ops.linear_bwd(down, H, dY[0], Ad[0], Bd[0], alpha, U=Ud)
    dX, dA, dB = ops.gated_bwd(qs, X[0], dH, GU, A[0], B[0], alpha, U=U)
    ref = oracle.gated_bwd(Ws, X[1], torch_to_f64(dH), torch_to_f64(GU), A[1], B[1], alpha, "silu")
    for got, want, name in zip((dX, dA, dB), ref, ("dX", "dA", "dB")):
        err = np.linalg.norm(torch_to_f64(got) - want) / np.linalg.norm(want)
        assert err <= (E if name != "dA" else 1e-5), (name, err)   # dB reads the rounded U


def test_captured_training_pass_follows_its_inputs():
    M, N, K, r = 70, 104, 192, 16
    qs, Ws, X, A, B, rng = block(13, M, N, K, r)
    dH = bf16(rng, (M, N))[0]
    x, dh = X[0].clone(), dH.clone()

    def step():
        H, GU, U = ops.gated_fwd(qs, x, A[0], B[0], 16.0, save=True)
        return (H,) + ops.gated_bwd(qs, x, dh, GU, A[0], B[0], 16.0, U=U)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for k in range(4):
        x.copy_(X[0] * (k + 1))
        dh.copy_(dH * (1 - 0.25 * k))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


def test_two_streams():
    M, N, K, r = 40, 512, 256, 16
    qs, Ws, X, A, B, rng = block(14, M, N, K, r)
    want = ops.gated_fwd(qs, X[0], A[0], B[0], 16.0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for k in range(6):
        with torch.cuda.stream(streams[k % 2]):
            got.append(ops.gated_fwd(qs, X[0], A[0], B[0], 16.0))
    torch.cuda.synchronize()
    for h in got:
        assert torch.equal(h, want)
