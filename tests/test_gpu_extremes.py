"""GPU: the adapter dropout and the 8-bit linears at the ends of their ranges
(element numbers past 2^32, operands near 2^31 elements), and used at once: two
streams, a backward captured while the same calls run eagerly.  Bounds as in
tests/test_gpu_dropout.py."""

import numpy as np
import pytest
import torch

from bit_quantized_finetuning_nf4_amd import ops, synth
from oracle import dropout as OD
from oracle import i8 as OI
from tests.helpers import bits_to_torch, torch_to_f64
from tests.test_gpu_dropout import E, F, adapter_bounds, bf16, make, within

pytestmark = pytest.mark.gpu


def test_dropout_past_2_32_elements_and_2_32_blocks():
    n = (1 << 35) + 4099   # 64 GiB, in place
    x = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    x.fill_(1.0)
    drop = ops.Dropout(0.25, 77, 3)
    ops.dropout(x, drop, out=x)
    torch.cuda.synchronize()
    one = float(np.float32(OD.keep_scale(0.25)))
    want = float(torch.tensor(one).to(torch.bfloat16))
    for first in (0, (1 << 31) - 64, (1 << 32) - 64, (1 << 34) + 8, (1 << 35) - 64, n - 4099):
        count = min(4099, n - first)
        keep = OD.keep_mask(count, 0.25, 77, 3, first=first)
        assert np.array_equal(torch_to_f64(x[first:first + count]), np.where(keep, want, 0.0)), first
    del x
    torch.cuda.empty_cache()


def test_linear_under_dropout_of_nearly_2_31_inputs():
    M, N, K, r, p, alpha = 524288, 64, 4032, 8, 0.2, 8.0   # M K = 2.11e9
    rng = np.random.default_rng(12)
    q = ops.quantize(bits_to_torch(synth.to_bf16_bits(rng.standard_normal((N, K)) * 0.02)))
    Wd = torch_to_f64(ops.dequant(q)).reshape(N, K)
    A, Ar = bf16(rng, (r, K), 0.1)
    B, Br = bf16(rng, (N, r), 0.1)
    rows = np.r_[0:130, M - 130:M]
    at = torch.from_numpy(rows).cuda()
    Xs, Xr = bf16(rng, (rows.size, K))
    dYs, dYr = bf16(rng, (rows.size, N))
    X = torch.ones((M, K), dtype=torch.bfloat16, device="cuda")
    dY = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    X[at], dY[at] = Xs, dYs
    drop = ops.Dropout(p, 9, 4)
    D = np.concatenate([OD.keep_mask(130 * K, p, 9, 4, first=int(f) * K).reshape(130, K) for f in (0, M - 130)])
    D = D * OD.keep_scale(p)
    Y, U = ops.linear_fwd(q, X, A, B, alpha, save_u=True, drop=drop)
    torch.cuda.synchronize()
    s, Ur = alpha / r, (D * Xr) @ Ar.T
    u_err = K * F * (np.abs(D * Xr) @ np.abs(Ar).T)
    within(U[at], Ur, 1.01 * (E * np.abs(Ur) + 2 * u_err), "U")
    Yr = Xr @ Wd.T + s * (Ur @ Br.T)
    tol = (E * np.abs(Yr) + (K + 34) * F * (np.abs(Xr) @ np.abs(Wd).T)
           + s * ((2.01 * E * np.abs(Ur) + 2 * u_err) @ np.abs(Br).T + (r + 34) * F * (np.abs(Ur) @ np.abs(Br).T)))
    within(Y[at], Yr, 1.01 * tol, "Y")
    dX, dA, dB = ops.linear_bwd(q, X, dY, A, B, alpha, U=U, drop=drop)
    torch.cuda.synchronize()
    # the rows without a gradient add exact zeros
    bounds = adapter_bounds(Xr, dYr, Ar, Br, Wd, s, D, torch_to_f64(U[at]))
    for g, (ref, t), name in zip((dX[at], dA, dB), bounds, ("dX", "dA", "dB")):
        within(g, ref, t, name)
    assert not dX[130:M - 130].any()


@pytest.mark.parametrize("M", [1, 20, 40, 300])
def test_i8_weight_of_nearly_2_31_codes(M):
    N, K, r = 131072, 16256, 8
    rng = np.random.default_rng(M)
    W = torch.empty((N, K), dtype=torch.bfloat16, device="cuda")
    W.fill_(0.01)
    last, lastr = bf16(rng, (200, K), 0.02)
    W[-200:] = last
    w = ops.i8_quantize(W)
    del W
    X, Xr = bf16(rng, (M, K))
    A, Ar = bf16(rng, (r, K), 0.1)
    B, Br = bf16(rng, (N, r), 0.1)
    Y = ops.i8_linear_fwd(w, X, A, B, 8.0)
    (wc, ws), (xc, sx) = OI.i8_quantize(lastr), OI.i8_quantize(Xr)
    main = OI.i8_matmul(xc, sx, wc, ws)
    Ur = Xr @ Ar.T
    u_err = K * F * (np.abs(Xr) @ np.abs(Ar).T)
    Bl = np.abs(Br[-200:])
    ref = main + Ur @ Br[-200:].T
    parts = 34 * 2.0**-24 * (np.abs(xc.astype(np.float64)) @ np.abs(wc.astype(np.float64)).T) * sx[:, None] * ws[None, :]
    tol = (E * np.abs(ref) + parts
           + (2.01 * E * np.abs(Ur) + 2 * u_err) @ Bl.T + (r + 34) * F * (np.abs(Ur) @ Bl.T))
    within(Y[:, -200:], ref, 1.01 * tol, "Y")
    del w, Y
    torch.cuda.empty_cache()


def test_two_streams_at_once():
    M, N, K, r = 300, 1024, 1088, 64
    d = make(M, N, K, r, 31)
    w = ops.i8_quantize(torch.randn(N, K, device="cuda").mul(0.02).to(torch.bfloat16))
    drop = ops.Dropout(0.3, 4, 5)

    def nf4():
        Y, U = ops.linear_fwd(d["q"], d["X"], d["A"], d["B"], 16.0, save_u=True, drop=drop)
        return (Y, U) + tuple(ops.linear_bwd(d["q"], d["X"], d["dY"], d["A"], d["B"], 16.0, U=U, drop=drop))

    def i8():
        Y, U = ops.i8_linear_fwd(w, d["X"], d["A"], d["B"], 16.0, save_u=True, drop=drop)
        return (Y, U) + tuple(ops.i8_linear_bwd(w, d["X"], d["dY"], d["A"], d["B"], 16.0, U=U, drop=drop))

    want_n, want_i = nf4(), i8()
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got_n, got_i = [], []
    for _ in range(5):
        with torch.cuda.stream(a):
            got_n.append(nf4())
        with torch.cuda.stream(b):
            got_i.append(i8())
    torch.cuda.synchronize()
    for got, want in [(g, want_n) for g in got_n] + [(g, want_i) for g in got_i]:
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("M", [1, 70, 1100])
def test_training_pass_captured_with_its_own_masks(M):
    """Forward and backward of both linears in one graph, whose masks follow a
    step count on the device, with the same calls run eagerly in between."""
    N, K, r = 264, 576, 24
    d = make(M, N, K, r, 17)
    w = ops.i8_quantize(torch.randn(N, K, device="cuda").mul(0.02).to(torch.bfloat16))
    step = torch.zeros(1, dtype=torch.int64, device="cuda")

    def both(drop):
        out = []
        Y, U = ops.linear_fwd(d["q"], d["X"], d["A"], d["B"], 16.0, save_u=True, drop=drop)
        out += [Y, U, *ops.linear_bwd(d["q"], d["X"], d["dY"], d["A"], d["B"], 16.0, U=U, drop=drop)]
        Y, U = ops.i8_linear_fwd(w, d["X"], d["A"], d["B"], 16.0, save_u=True, drop=drop)
        out += [Y, U, *ops.i8_linear_bwd(w, d["X"], d["dY"], d["A"], d["B"], 16.0, U=U, drop=drop)]
        return out

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(ops.Dropout(0.3, 21, 100, step))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = both(ops.Dropout(0.3, 21, 100, step))
    seen = []
    for k in (0, 3, 1, 3):
        step.fill_(k)
        g.replay()
        torch.cuda.synchronize()
        want = both(ops.Dropout(0.3, 21, 100 + k))
        assert all(torch.equal(x, y) for x, y in zip(got, want)), k
        seen.append(got[1].clone())
    assert not torch.equal(seen[0], seen[1]) and torch.equal(seen[1], seen[3])
