"""GPU: the middling products in every tile shape, split and unsplit, with each
adapter term.  The sizes are the smallest found at which the choice by
estimated time takes the shape named (on 256 CUs; on another card they are
still a sweep of sizes).  Bounds as in tests/test_gpu_dropout.py."""

import numpy as np
import pytest
import torch

import oracle
from bit_quantized_finetuning_nf4_amd import ops, synth
from oracle import dropout as OD
from oracle import i8 as OI
from tests.helpers import bits_to_torch, torch_to_f64
from tests.test_gpu_dropout import E, F, adapter_bounds, bf16, within

pytestmark = pytest.mark.gpu

# tokens, channels of the product, 128-byte lines of its contraction
SIZES = {
    "64x64": (49, 64, 1), "64x64 split": (43, 64, 16), "64x128": (66, 9024, 1), "64x128 split": (67, 2816, 55),
    "128x128": (135, 11392, 6), "128x128 split": (65, 9280, 45), "192x128": (324, 11456, 17),
    "192x128 split": (129, 5696, 54), "256x128": (386, 10944, 1), "128x128 of one line": (271, 6656, 1),
    "256x192": (548, 11008, 1),
    "256x256": (1062, 10560, 2), "256x256 split": (195, 8512, 71),
}


@pytest.mark.parametrize("name", SIZES)
@pytest.mark.parametrize("r,p", [(0, 0.0), (24, 0.0), (24, 0.3), (64, 0.1), (96, 0.2), (128, 0.0), (128, 0.6)])
def test_dx(name, r, p):
    M, K, lines = SIZES[name]
    N = 64 * lines
    print(f"[tiles dX] {name} M{M} N{N} K{K} r{r} p{p}", flush=True)
    rng = np.random.default_rng(M + r)
    w = ops.i8_quantize(bf16(rng, (N, K), 0.02)[0])
    Wd = torch_to_f64(ops.i8_dequant(w))
    dY, dYr = bf16(rng, (M, N))
    if r == 0:
        got = ops.i8_linear_bwd(w, None, dY)[0]
        ref = dYr @ Wd
        within(got, ref, 1.01 * (E * np.abs(ref) + N * F * (np.abs(dYr) @ np.abs(Wd))), "dX")
        return
    X, Xr = bf16(rng, (M, K))
    A, Ar = bf16(rng, (r, K), 0.1)
    B, Br = bf16(rng, (N, r), 0.1)
    U, Ur = bf16(rng, (M, r))
    drop = ops.Dropout(p, 31, 7) if p > 0 else None
    D = OD.keep_mask(M * K, p, 31, 7).reshape(M, K) * OD.keep_scale(p)
    got = ops.i8_linear_bwd(w, X, dY, A, B, 16.0, U=U, drop=drop)
    for g, (ref, tol), what in zip(got, adapter_bounds(Xr, dYr, Ar, Br, Wd, 16.0 / r, D, Ur), ("dX", "dA", "dB")):
        within(g, ref, tol, what)


@pytest.mark.parametrize("name", SIZES)
@pytest.mark.parametrize("r", [0, 24, 64, 128])
def test_i8_forward(name, r):
    M, N, lines = SIZES[name]
    K = 128 * lines
    print(f"[tiles i8] {name} M{M} N{N} K{K} r{r}", flush=True)
    rng = np.random.default_rng(M + r)
    W, Wr = bf16(rng, (N, K), 0.02)
    X, Xr = bf16(rng, (M, K))
    (wc, ws), (xc, sx) = OI.i8_quantize(Wr), OI.i8_quantize(Xr)
    main = OI.i8_matmul(xc, sx, wc, ws)
    w = ops.i8_quantize(W)
    # a split product adds fp32 parts, each of them rounded: 34 roundings of what the parts' magnitudes sum to
    parts = 34 * 2.0**-24 * (np.abs(xc.astype(np.float64)) @ np.abs(wc.astype(np.float64)).T) * sx[:, None] * ws[None, :]
    if r == 0:
        within(ops.i8_linear_fwd(w, X), main, 1.01 * (E * np.abs(main) + parts), "Y")
        return
    A, Ar = bf16(rng, (r, K), 0.1)
    B, Br = bf16(rng, (N, r), 0.1)
    Y, U = ops.i8_linear_fwd(w, X, A, B, 16.0, save_u=True)
    s, Ur = 16.0 / r, Xr @ Ar.T
    u_err = K * F * (np.abs(Xr) @ np.abs(Ar).T)
    within(U, Ur, 1.01 * (E * np.abs(Ur) + 2 * u_err), "U")
    ref = main + s * (Ur @ Br.T)
    tol = (E * np.abs(ref) + parts
           + s * ((2.01 * E * np.abs(Ur) + 2 * u_err) @ np.abs(Br).T + (r + 34) * F * (np.abs(Ur) @ np.abs(Br).T)))
    within(Y, ref, 1.01 * tol, "Y")


# up to 32 tokens: the streaming kernel in its widths, batches whole and partial, rounds whole and partial; and where
# tiles, split or not, take over
FEW = [(1, 1024, 8072), (2, 6152, 8192), (7, 4096, 16264), (8, 8200, 1160), (9, 16392, 2048), (16, 8192, 8072),
       (11, 28680, 640), (16, 4104, 1000), (17, 1000, 2968), (24, 4096, 4096), (32, 4104, 3000), (20, 8192, 1960),
       (1, 256, 22016), (8, 13824, 5120), (16, 5120, 13824), (16, 264, 22016), (20, 512, 8192), (32, 1024, 1024),
       (32, 5128, 5120), (24, 11008, 4096), (32, 16392, 4096)]


@pytest.mark.parametrize("M,N,K", FEW)
@pytest.mark.parametrize("r", [0, 40])
def test_i8_forward_of_few_tokens(M, N, K, r):
    print(f"[few i8] M{M} N{N} K{K} r{r}", flush=True)
    rng = np.random.default_rng(M + N + r)
    W, Wr = bf16(rng, (N, K), 0.02)
    X, Xr = bf16(rng, (M, K))
    (wc, ws), (xc, sx) = OI.i8_quantize(Wr), OI.i8_quantize(Xr)
    main = OI.i8_matmul(xc, sx, wc, ws)
    w = ops.i8_quantize(W)
    # without a workspace nothing is split: the exact sum, the scales' product and their product rounded
    within(ops.i8_matmul(ops.i8_quantize(X), w), main, 1.01 * (E + 3.01 * 2.0**-24) * np.abs(main), "matmul")
    parts = 34 * 2.0**-24 * (np.abs(xc.astype(np.float64)) @ np.abs(wc.astype(np.float64)).T) * sx[:, None] * ws[None, :]
    if r == 0:
        within(ops.i8_linear_fwd(w, X), main, 1.01 * (E * np.abs(main) + parts), "Y")
        return
    A, Ar = bf16(rng, (r, K), 0.1)
    B, Br = bf16(rng, (N, r), 0.1)
    Y, U = ops.i8_linear_fwd(w, X, A, B, 16.0, save_u=True)
    s, Ur = 16.0 / r, Xr @ Ar.T
    u_err = K * F * (np.abs(Xr) @ np.abs(Ar).T)
    within(U, Ur, 1.01 * (E * np.abs(Ur) + 2 * u_err), "U")
    ref = main + s * (Ur @ Br.T)
    tol = (E * np.abs(ref) + parts
           + s * ((2.01 * E * np.abs(Ur) + 2 * u_err) @ np.abs(Br).T + (r + 34) * F * (np.abs(Ur) @ np.abs(Br).T)))
    within(Y, ref, 1.01 * tol, "Y")


@pytest.mark.parametrize("name", SIZES)
def test_nf4_forward_under_dropout(name):
    M, N, lines = SIZES[name]
    K, r, p = 64 * lines, 24, 0.25
    print(f"[tiles nf4] {name} M{M} N{N} K{K}", flush=True)
    rng = np.random.default_rng(M)
    q = ops.quantize(bits_to_torch(synth.to_bf16_bits(rng.standard_normal((N, K)) * 0.02)))
    Wd = torch_to_f64(ops.dequant(q)).reshape(N, K)
    X, Xr = bf16(rng, (M, K))
    A, Ar = bf16(rng, (r, K), 0.1)
    B, Br = bf16(rng, (N, r), 0.1)
    Y, U = ops.linear_fwd(q, X, A, B, 16.0, save_u=True, drop=ops.Dropout(p, 5, 6))
    D = OD.keep_mask(M * K, p, 5, 6).reshape(M, K) * OD.keep_scale(p)
    s, Ur = 16.0 / r, (D * Xr) @ Ar.T
    u_err = K * F * (np.abs(D * Xr) @ np.abs(Ar).T)
    within(U, Ur, 1.01 * (E * np.abs(Ur) + 2 * u_err), "U")
    ref = Xr @ Wd.T + s * (Ur @ Br.T)
    tol = (E * np.abs(ref) + (K + 34) * F * (np.abs(Xr) @ np.abs(Wd).T)
           + s * ((2.01 * E * np.abs(Ur) + 2 * u_err) @ np.abs(Br).T + (r + 34) * F * (np.abs(Ur) @ np.abs(Br).T)))
    within(Y, ref, 1.01 * tol, "Y")


@pytest.mark.parametrize("name", ["64x64", "256x128", "256x192", "256x256", "256x256 split"])
@pytest.mark.parametrize("r", [40, 64, 96, 128])
def test_an_infinite_gradient_stays_in_its_row(name, r):
    M, K, lines = SIZES[name]
    N = 64 * lines
    print(f"[tiles inf] {name} M{M} N{N} K{K} r{r}", flush=True)
    rng = np.random.default_rng(M + r)
    w = ops.i8_quantize(bf16(rng, (N, K), 0.02)[0])
    X, A, B = bf16(rng, (M, K))[0], bf16(rng, (r, K), 0.1)[0], bf16(rng, (N, r), 0.1)[0]
    dY = bf16(rng, (M, N))[0]
    drop = ops.Dropout(0.3, 31, 7)
    want = ops.i8_linear_bwd(w, X, dY, A, B, 16.0, drop=drop)[0]
    dY[7, 0] = float("inf")
    got = ops.i8_linear_bwd(w, X, dY, A, B, 16.0, drop=drop)[0]
    rest = [i for i in range(M) if i != 7]
    assert torch.equal(got[rest], want[rest])
    assert not got[7].isfinite().any()
