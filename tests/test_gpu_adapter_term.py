"""GPU: the adapter's term alone, in every product kernel.

The frozen weight is zero, so Y is s U B^T and dX is s drop'(G A), rounded
once.  X, A, dY and B hold small integers, so U and G are exact in fp32
whatever the order of their sums (below 2^24), and what is left is
  - s and the dropout's scale applied in fp32: 2^-24 each;
  - two bf16 parts: 2^-8 of the value after the first, 2^-16 after the second;
  - the sum of 2 r fp32 products: 2^-23 each of the sum of their magnitudes;
  - the result's own rounding: 2^-8 of it.
A side operand rounded to bf16 (2^-8 of every product) is far outside that
wherever the products cancel.
"""

import numpy as np
import pytest
import torch

from bit_quantized_finetuning_nf4_amd import _lib, ops
from oracle import dropout as OD
from tests.test_gpu_dropout import within
from tests.test_gpu_tiles import SIZES

pytestmark = pytest.mark.gpu

E = 2.0**-8
ALPHA = 10.0   # s is a power of two at no rank here


def ints(rng, shape, top=8):
    """(GPU bf16 tensor, fp64) of integers in [-top, top]."""
    x = rng.integers(-top, top + 1, shape).astype(np.float64)
    return torch.from_numpy(x).to(torch.bfloat16).cuda(), x


def term_tol(ref, T, W, r):
    """Bound of ref = T W from the parts of T: T [M x r], W [r x N]."""
    return 1.001 * (E * np.abs(ref) + (2.0**-16 + 2 * 2.0**-24 + 2 * r * 2.0**-23) * (np.abs(T) @ np.abs(W)))


def check_forward(run, rng, M, N, K, r, p, alpha=ALPHA):
    X, Xr = ints(rng, (M, K))
    A, Ar = ints(rng, (r, K))
    B, Br = ints(rng, (N, r))
    drop = ops.Dropout(p, 31, 7) if p > 0 else None
    keep = OD.keep_mask(M * K, p, 31, 7).reshape(M, K) if p > 0 else 1.0
    S = (Xr * keep) @ Ar.T
    assert np.abs(S).max() < 2**24 and (np.abs(Xr * keep) @ np.abs(Ar).T).max() < 2**24
    Ur = S * (OD.keep_scale(p) if p > 0 else 1.0)
    Y, U = run(X, A, B, drop)
    within(U, Ur, 1.001 * (E + 2.0**-24) * np.abs(Ur), "U")
    T = alpha / r * Ur
    within(Y, T @ Br.T, term_tol(T @ Br.T, T, Br.T, r), "Y")


@pytest.mark.parametrize("name", SIZES)
@pytest.mark.parametrize("r", [24, 64, 96, 128])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_dx(name, r, p):
    M, K, lines = SIZES[name]
    N = 64 * lines
    print(f"[term dX] {name} M{M} N{N} K{K} r{r} p{p}", flush=True)
    rng = np.random.default_rng(M + r)
    w = ops.i8_quantize(torch.zeros((N, K), dtype=torch.bfloat16, device="cuda"))
    dY, dYr = ints(rng, (M, N))
    X = ints(rng, (M, K))[0]
    A, Ar = ints(rng, (r, K))
    B, Br = ints(rng, (N, r))
    G = dYr @ Br
    assert (np.abs(dYr) @ np.abs(Br)).max() < 2**24
    drop = ops.Dropout(p, 31, 7) if p > 0 else None
    D = OD.keep_mask(M * K, p, 31, 7).reshape(M, K) * OD.keep_scale(p) if p > 0 else 1.0
    U = torch.zeros((M, r), dtype=torch.bfloat16, device="cuda")
    dX = ops.i8_linear_bwd(w, X, dY, A, B, ALPHA, U=U, drop=drop)[0]
    T = ALPHA / r * G
    ref = D * (T @ Ar)
    tol = term_tol(T @ Ar, T, Ar, r)
    within(dX, ref, D * tol, "dX")


@pytest.mark.parametrize("name", SIZES)
@pytest.mark.parametrize("r", [24, 64, 96, 128])
def test_i8_forward(name, r):
    M, N, lines = SIZES[name]
    K = 128 * lines
    print(f"[term i8] {name} M{M} N{N} K{K} r{r}", flush=True)
    w = ops.i8_quantize(torch.zeros((N, K), dtype=torch.bfloat16, device="cuda"))
    check_forward(lambda X, A, B, drop: ops.i8_linear_fwd(w, X, A, B, ALPHA, save_u=True, drop=drop),
                  np.random.default_rng(M + r), M, N, K, r, 0.0)


# up to 32 tokens: each width of the streaming kernel, and tiles
@pytest.mark.parametrize("M,N,K", [(1, 1024, 8072), (16, 8192, 384), (20, 4096, 2056), (30, 16392, 1032), (32, 1024, 1024)])
@pytest.mark.parametrize("r,p", [(8, 0.0), (24, 0.3), (96, 0.0), (128, 0.3)])
def test_i8_forward_of_few_tokens(M, N, K, r, p):
    print(f"[term few] M{M} N{N} K{K} r{r} p{p}", flush=True)
    w = ops.i8_quantize(torch.zeros((N, K), dtype=torch.bfloat16, device="cuda"))
    check_forward(lambda X, A, B, drop: ops.i8_linear_fwd(w, X, A, B, ALPHA, save_u=True, drop=drop),
                  np.random.default_rng(M + r), M, N, K, r, p)


# the staged path, and (with room for no bf16 weight) the fused one: whole rounds of tiles, and a last round in halves
@pytest.mark.parametrize("M,N,K", [(70, 1032, 1088), (300, 256 * 130, 64), (263, 520, 4096)])
@pytest.mark.parametrize("r", [24, 64, 128])
@pytest.mark.parametrize("fused", [False, True])
def test_nf4_forward(M, N, K, r, fused):
    print(f"[term nf4] M{M} N{N} K{K} r{r} fused {fused}", flush=True)
    q = ops.quantize(torch.zeros((N, K), dtype=torch.bfloat16, device="cuda"))
    nbytes = ops.workspace_bytes(_lib.QLORA_OP_FWD_DROP, M, N, K, r)
    if fused and nbytes > 2 * N * K:
        nbytes -= 2 * N * K
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    check_forward(lambda X, A, B, drop: ops.linear_fwd(q, X, A, B, ALPHA, save_u=True, drop=drop, ws=ws),
                  np.random.default_rng(M + r), M, N, K, r, 0.25)


@pytest.mark.parametrize("name", ["256x128", "256x192", "256x256", "256x256 split"])
@pytest.mark.parametrize("r", [24, 128])
def test_nf4_forward_in_wide_tiles(name, r):
    M, N, lines = SIZES[name]
    K = 64 * lines
    print(f"[term nf4] {name} M{M} N{N} K{K} r{r}", flush=True)
    q = ops.quantize(torch.zeros((N, K), dtype=torch.bfloat16, device="cuda"))
    check_forward(lambda X, A, B, drop: ops.linear_fwd(q, X, A, B, ALPHA, save_u=True, drop=drop),
                  np.random.default_rng(M + r), M, N, K, r, 0.25)


def test_u_saved_or_not_gives_the_same():
    rng = np.random.default_rng(3)
    for M, N, K, r in ((5, 264, 512, 16), (300, 1032, 1088, 64), (1100, 520, 576, 24)):
        W = torch.randn((N, K), device="cuda").mul_(0.02).to(torch.bfloat16)
        X, A, B = ints(rng, (M, K))[0], ints(rng, (r, K))[0], ints(rng, (N, r))[0]
        drop = ops.Dropout(0.2, 3, 4)
        for fwd, w in ((ops.linear_fwd, ops.quantize(W)), (ops.i8_linear_fwd, ops.i8_quantize(W))):
            Y, U = fwd(w, X, A, B, ALPHA, save_u=True, drop=drop)
            assert torch.equal(fwd(w, X, A, B, ALPHA, drop=drop), Y)


@pytest.mark.parametrize("M,N,K,r", [(5, 264, 512, 16), (300, 1032, 1088, 64), (1100, 520, 576, 24)])
def test_alpha_of_zero_and_below(M, N, K, r):
    rng = np.random.default_rng(M)
    W = torch.from_numpy(rng.standard_normal((N, K)) * 0.02).to(torch.bfloat16).cuda()
    X, dY = ints(rng, (M, K))[0], ints(rng, (M, N))[0]
    A, B = ints(rng, (r, K))[0], ints(rng, (N, r))[0]
    w = ops.i8_quantize(W)
    drop = ops.Dropout(0.2, 3, 4)
    assert torch.equal(ops.i8_linear_fwd(w, X, A, B, 0.0, drop=drop), ops.i8_linear_fwd(w, X))
    none = ops.i8_linear_bwd(w, None, dY)[0]
    U = torch.ones((M, r), dtype=torch.bfloat16, device="cuda")
    dX, dA, dB = ops.i8_linear_bwd(w, X, dY, A, B, 0.0, U=U, drop=drop)
    assert torch.equal(dX, none) and bool((dA == 0).all()) and bool((dB == 0).all())
    # -alpha: the gradients with the other sign (each sum off by 3 M products' 2^-23 at most: a matrix instruction's
    # rounding need not be the same for a sum and its negative), and the forward's term
    plus, minus = (ops.i8_linear_bwd(w, X, dY, A, B, a, U=U, drop=drop) for a in (ALPHA, -ALPHA))
    G = ALPHA / r * (dY.double().abs() @ B.double().abs())
    assert bool(((plus[1] + minus[1]).abs() <= 2 * 3 * M * 2.0**-23 * (G.T @ X.double().abs()) * 1.3).all())
    dB = ALPHA / r * (dY.double().abs().T @ U.double())
    assert bool(((plus[2] + minus[2]).abs() <= 2 * M * 2.0**-23 * dB).all())
    zero, q = ops.i8_quantize(torch.zeros_like(W)), ops.quantize(torch.zeros_like(W))
    for fwd, z in ((ops.i8_linear_fwd, zero), (ops.linear_fwd, q)):
        check_forward(lambda X, A, B, drop: fwd(z, X, A, B, -ALPHA, save_u=True, drop=drop), rng, M, N, K, r, 0.25, -ALPHA)
