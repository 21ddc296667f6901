"""GPU: the linear under dropout on the other codebooks, the FP8 second level,
and weights whose bf16 form is larger than the last-level cache (dequantized in
reverse order). The adapter's last step rides with the dequantization there.

Inputs of small integers against the weight that ops.dequant gives, whose
levels are no integers: one column of X, or one row of dY, per output is not
zero, so each product is one number and the result exact."""

import numpy as np
import pytest
import torch

from bit_quantized_finetuning_nf4_amd import ops
from oracle import dropout as OD

pytestmark = pytest.mark.gpu


def gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).cuda()


def picks(rng, rows, cols):
    """[rows x cols] zeros with a one in each row, and where."""
    at = rng.integers(0, cols, rows)
    x = np.zeros((rows, cols))
    x[np.arange(rows), at] = 1.0
    return x, at


@pytest.mark.parametrize("codebook", ["nf4", "fp4", "int4"])
@pytest.mark.parametrize("absmax", ["linear", "fp8"])
@pytest.mark.parametrize("M,N,K,r", [(70, 264, 576, 16), (1030, 520, 1088, 64)])
def test_codebooks(codebook, absmax, M, N, K, r):
    print(f"[drop codebook] {codebook} {absmax} M{M} N{N} K{K} r{r}", flush=True)
    rng = np.random.default_rng(M + r)
    q = ops.quantize(gpu(rng.standard_normal((N, K)) * 0.02), codebook=codebook, absmax_format=absmax)
    Wd = ops.dequant(q).double().cpu().numpy()
    drop = ops.Dropout(0.5, 5, 6)
    D = 2.0 * OD.keep_mask(M * K, 0.5, 5, 6).reshape(M, K)
    X, at = picks(rng, M, K)
    # the adapter sees X too; A and B of ones and a term of whole 1/64s, larger than any level's last bit
    A, B = rng.choice([-1.0, 1.0], (r, K)), rng.integers(-1, 2, (N, r)).astype(np.float64)
    Y, U = ops.linear_fwd(q, gpu(X), gpu(A), gpu(B), r / 64.0, save_u=True, drop=drop)
    Ur = (D * X) @ A.T
    assert torch.equal(U.cpu(), torch.from_numpy(Ur).to(torch.bfloat16))
    # fp32 adds a level to the term once: half a step of it, then bf16's
    ref = Wd[:, at].T + Ur @ B.T / 64.0
    err = np.abs(Y.double().cpu().numpy() - ref)
    assert (err <= 1.001 * (2.0**-8 * np.abs(ref) + 2.0**-24 * (np.abs(Wd[:, at].T) + 2 * r / 64.0))).all()
    dY, at = picks(rng, M, N)
    Z = torch.zeros((M, r), dtype=torch.bfloat16, device="cuda")
    dX, dA, dB = ops.linear_bwd(q, gpu(X), gpu(dY), gpu(A), gpu(B), r / 64.0, U=Z, drop=drop)
    G = dY @ B
    ref = Wd[at] + D * (G @ A) / 64.0
    err = np.abs(dX.double().cpu().numpy() - ref)
    assert (err <= 1.001 * (2.0**-8 * np.abs(ref) + 2.0**-24 * (np.abs(Wd[at]) + 2 * r / 64.0))).all()
    assert torch.equal(dA.cpu(), torch.from_numpy(G.T @ (D * X) / 64.0).float()) and bool((dB == 0).all())


@pytest.mark.parametrize("kind", ["nf4", "i8"])
def test_weights_past_the_last_level_cache(kind):
    M, N, K, r = 1030, 16392, 8256, 16   # 271 MB in bf16, N % 64 != 0
    print(f"[drop large] {kind} M{M} N{N} K{K} r{r}", flush=True)
    rng = np.random.default_rng(3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    W = torch.randn((N, K), generator=gen, device="cuda").mul_(0.02).to(torch.bfloat16)
    if kind == "nf4":
        w, fwd, bwd = ops.quantize(W), ops.linear_fwd, ops.linear_bwd
        Wd = ops.dequant(w).view(N, K)
    else:
        w, fwd, bwd = ops.i8_quantize(W), ops.i8_linear_fwd, ops.i8_linear_bwd
        Wd = ops.i8_dequant(w)
    drop = ops.Dropout(0.5, 5, 6)
    D = torch.from_numpy(2.0 * OD.keep_mask(M * K, 0.5, 5, 6).reshape(M, K)).cuda()
    X, at = picks(rng, M, K)
    A, B = rng.choice([-1.0, 1.0], (r, K)), rng.integers(-1, 2, (N, r)).astype(np.float64)
    At, Bt, Xt = (torch.from_numpy(v).cuda() for v in (A, B, X))
    if kind == "nf4":
        Y, U = fwd(w, gpu(X), gpu(A), gpu(B), r / 64.0, save_u=True, drop=drop)
        Ur = (D * Xt) @ At.T
        assert torch.equal(U, Ur.to(torch.bfloat16))
        main = Wd[:, torch.from_numpy(at).cuda()].T.double()
        ref = main + Ur @ Bt.T / 64.0
        tol = 1.001 * (2.0**-8 * ref.abs() + 2.0**-24 * (main.abs() + 2 * r / 64.0))
        assert bool(((Y.double() - ref).abs() <= tol).all())
    dY, at = picks(rng, M, N)
    at = torch.from_numpy(at).cuda()
    Z = torch.zeros((M, r), dtype=torch.bfloat16, device="cuda")
    dX, dA, dB = bwd(w, gpu(X), gpu(dY), gpu(A), gpu(B), r / 64.0, U=Z, drop=drop)
    G = torch.from_numpy(dY).cuda() @ Bt
    main = Wd[at].double()
    ref = main + D * (G @ At) / 64.0
    tol = 1.001 * (2.0**-8 * ref.abs() + 2.0**-24 * (main.abs() + 2 * r / 64.0))
    assert bool(((dX.double() - ref).abs() <= tol).all())
    assert torch.equal(dA, (G.T @ (D * Xt) / 64.0).float()) and bool((dB == 0).all())
