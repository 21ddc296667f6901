"""GPU: dropout and the NF4 linear with its adapter under dropout.

Tolerances are bounds, element by element.  bf16 rounds by at most E = 2^-8
of the value, fp32 by 2^-24; a sum of n fp32 products in any order is off by
at most n 2^-23 of the sum of their magnitudes (n additions and n products,
2^-24 each).
"""

import numpy as np
import pytest
import torch

import oracle
from bit_quantized_finetuning_nf4_amd import _lib, ops, synth
from oracle import dropout as OD
from tests.helpers import bits_to_torch, torch_to_bits, torch_to_f64

pytestmark = pytest.mark.gpu

E = 2.0**-8
F = 2.0**-23


def bf16(rng, shape, std=1.0):
    """(GPU tensor, its values in fp64)."""
    bits = synth.to_bf16_bits(rng.standard_normal(shape) * std)
    return bits_to_torch(bits), oracle.bf16_bits_to_f64(bits).reshape(shape)


def within(got, ref, tol, name):
    got = torch_to_f64(got)
    assert np.isfinite(got).all(), name
    over = np.abs(got - ref) - (tol + 1e-37)
    assert (over <= 0).all(), f"{name}: {over.max():.3e} over its bound, {(over > 0).sum()} of {over.size}"


def adapter_bounds(X, dY, A, B, Wd, s, D, U):
    """(dX, dA, dB) and their bounds; D: the kept scale of every element of X
    (0 where dropped), U: the bf16 values handed to the backward.  G is bf16
    in dX, fp32 (three bf16 parts, 2^-24) in dA, plus its own sum's error."""
    M, N, K, r = X.shape[0], dY.shape[1], X.shape[1], A.shape[0]
    G = dY @ B
    Gm = np.abs(dY) @ np.abs(B)
    g_err = N * F * Gm
    dX = dY @ Wd + s * D * (G @ A)
    # s G may be rounded to bf16 once more where nothing is masked
    tail = s * D * ((2.01 * E * np.abs(G) + 2 * g_err) @ np.abs(A) + r * F * (np.abs(G) @ np.abs(A)))
    dX_tol = 1.01 * (E * np.abs(dX) + N * F * (np.abs(dY) @ np.abs(Wd)) + tail)
    XD = D * X
    dA = s * (G.T @ XD)
    dA_tol = 1.01 * s * ((2.0**-24 * np.abs(G) + g_err).T @ np.abs(XD) + 3 * M * F * (np.abs(G).T @ np.abs(XD)))
    dB = s * (dY.T @ U)
    dB_tol = 1.01 * s * M * F * (np.abs(dY).T @ np.abs(U))
    return (dX, dX_tol), (dA, dA_tol), (dB, dB_tol)


# --- elementwise -----------------------------------------------------------

def expect_dropout(x_bits, p, seed, offset):
    """bf16 bits: one fp32 product, rounded to bf16; 0 where dropped."""
    scale = np.float32(OD.keep_scale(p))
    y = oracle.f32_to_bf16_bits(oracle.bf16_bits_to_f32(x_bits) * scale)
    keep = OD.keep_mask(x_bits.size, p, seed, offset).reshape(x_bits.shape)
    return np.where(keep, y, 0).astype(np.uint16)


@pytest.mark.parametrize("n", [1, 7, 8, 9, 63, 1024, 8191, 8192, 8193, 32768 + 5, 1 << 20])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.999])
def test_dropout_bits(n, p):
    print(f"[dropout] n={n} p={p}", flush=True)
    bits = synth.to_bf16_bits(np.random.default_rng(n).standard_normal(n))
    drop = ops.Dropout(p, seed=0x123456789ABCDEF0, offset=0xFEDCBA9876543210)
    y = ops.dropout(bits_to_torch(bits), drop)
    assert np.array_equal(torch_to_bits(y), expect_dropout(bits, p, drop.seed, drop.offset))


def test_dropout_in_place_shape_and_no_neighbours():
    bits = synth.to_bf16_bits(np.random.default_rng(1).standard_normal((3, 5, 7)))
    whole = torch.full((105 + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
    x = whole[:105].view(3, 5, 7)
    x.copy_(bits_to_torch(bits).view(3, 5, 7))
    drop = ops.Dropout(0.25, 9, 1)
    y = ops.dropout(x, drop, out=x)
    assert y.data_ptr() == x.data_ptr() and y.shape == (3, 5, 7)
    assert np.array_equal(torch_to_bits(y), expect_dropout(bits, 0.25, 9, 1))
    assert (whole[105:] == 3.0).all()
    assert ops.dropout(whole[:0], drop).numel() == 0


def test_dropped_infinities_and_nans_are_zero():
    n = 4096
    keep = OD.keep_mask(n, 0.5, 3, 4)
    x = torch.full((n,), float("nan"), dtype=torch.bfloat16, device="cuda")
    x[1::2] = float("inf")
    y = torch_to_f64(ops.dropout(x, ops.Dropout(0.5, 3, 4)))
    assert (y[~keep] == 0).all()
    assert np.isnan(y[keep & (np.arange(n) % 2 == 0)]).all() and np.isinf(y[keep & (np.arange(n) % 2 == 1)]).all()


def test_far_blocks_use_the_high_counter_word():
    """Element numbers above 2^32 * 8 cannot be allocated as bf16 cheaply here;
    the offset's high word shares the same path, and a large flat tensor
    covers block numbers past 2^24."""
    n = (1 << 27) + 24
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    y = ops.dropout(x, ops.Dropout(0.5, 11, 1 << 40))
    tail = 4096 + 24
    want = OD.keep_mask(tail, 0.5, 11, 1 << 40, first=n - tail)
    assert np.array_equal(torch_to_f64(y[-tail:]) != 0, want)


def test_step_on_the_device_and_graph_replays():
    x = torch.randn(10000, device="cuda").to(torch.bfloat16)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    drop = ops.Dropout(0.3, 21, 100, step)
    out = torch.empty_like(x)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        ops.dropout(x, drop, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        ops.dropout(x, drop, out=out)
    bits = torch_to_bits(x)
    for k in (0, 1, 5, 2):
        step.fill_(k)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(torch_to_bits(out), expect_dropout(bits, 0.3, 21, 100 + k)), k
        eager = ops.dropout(x, ops.Dropout(0.3, 21, 100 + k))
        assert torch.equal(eager.view(torch.int16), out.view(torch.int16))


# --- the NF4 linear ----------------------------------------------------------

SHAPES = [
    # M, N, K, r, p
    (1, 64, 64, 8, 0.5),
    (70, 192, 320, 8, 0.1),
    (256, 1024, 1024, 16, 0.1),
    (300, 1032, 1088, 64, 0.3),     # N % 64 != 0: padded contraction in dX
    (513, 264, 320, 128, 0.05),     # the largest rank
    (130, 520, 576, 96, 0.4),       # rank of three chunks
    (1100, 776, 576, 24, 0.2),      # staged forward, rank with a partial chunk
    (1300, 832, 2112, 32, 0.6),
    (2048, 1088, 5120, 64, 0.05),   # narrower dX tiles
    (33, 8, 64, 8, 0.9),
]


def make(M, N, K, r, seed, ab=0.1):
    rng = np.random.default_rng(seed)
    q = ops.quantize(bits_to_torch(synth.to_bf16_bits(rng.standard_normal((N, K)) * 0.02)))
    Wd = torch_to_f64(ops.dequant(q)).reshape(N, K)
    d = dict(q=q, Wd=Wd)
    for name, shape, std in (("X", (M, K), 1.0), ("A", (r, K), ab), ("B", (N, r), ab), ("dY", (M, N), 1.0)):
        d[name], d[name + "r"] = bf16(rng, shape, std)
    return d


@pytest.mark.parametrize("M,N,K,r,p", SHAPES)
def test_linear_under_dropout(M, N, K, r, p):
    print(f"[linear drop] M{M} N{N} K{K} r{r} p{p}", flush=True)
    d = make(M, N, K, r, M + N + K + r)
    X, A, B, dY, Wd = d["Xr"], d["Ar"], d["Br"], d["dYr"], d["Wd"]
    drop = ops.Dropout(p, seed=17 + M, offset=5)
    s = 16.0 / r
    D = OD.keep_mask(M * K, p, drop.seed, 5).reshape(M, K) * OD.keep_scale(p)
    Y, U = ops.linear_fwd(d["q"], d["X"], d["A"], d["B"], 16.0, save_u=True, drop=drop)
    torch.cuda.synchronize()
    Ur = (D * X) @ A.T
    u_err = K * F * (np.abs(D * X) @ np.abs(A).T)
    within(U, Ur, 1.01 * (E * np.abs(Ur) + 2 * u_err), "U")
    Yr = X @ Wd.T + s * (Ur @ B.T)
    y_tol = (E * np.abs(Yr) + K * F * (np.abs(X) @ np.abs(Wd).T)
             + s * ((2.01 * E * np.abs(Ur) + 2 * u_err) @ np.abs(B).T + r * F * (np.abs(Ur) @ np.abs(B).T)))
    within(Y, Yr, 1.01 * y_tol, "Y")

    got = ops.linear_bwd(d["q"], d["X"], dY=d["dY"], A=d["A"], B=d["B"], alpha=16.0, U=U, drop=drop)
    torch.cuda.synchronize()
    for g, (ref, tol), name in zip(got, adapter_bounds(X, dY, A, B, Wd, s, D, torch_to_f64(U)), ("dX", "dA", "dB")):
        within(g, ref, tol, name)


def test_backward_recomputes_u_and_skips_dx():
    M, N, K, r = 200, 320, 448, 16
    d = make(M, N, K, r, 4)
    drop = ops.Dropout(0.25, 8, 1)
    _, U = ops.linear_fwd(d["q"], d["X"], d["A"], d["B"], 16.0, save_u=True, drop=drop)
    a = ops.linear_bwd(d["q"], d["X"], d["dY"], d["A"], d["B"], 16.0, U=U, drop=drop)
    b = ops.linear_bwd(d["q"], d["X"], d["dY"], d["A"], d["B"], 16.0, drop=drop)
    c = ops.linear_bwd(d["q"], d["X"], d["dY"], d["A"], d["B"], 16.0, U=U, need_dx=False, drop=drop)
    assert c[0] is None
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    for x, y in zip(a[1:], c[1:]):
        assert torch.equal(x, y)


def test_p_zero_is_the_plain_linear():
    d = make(300, 320, 448, 16, 6)
    Y0, U0 = ops.linear_fwd(d["q"], d["X"], d["A"], d["B"], 16.0, save_u=True)
    Y1, U1 = ops.linear_fwd(d["q"], d["X"], d["A"], d["B"], 16.0, save_u=True, drop=ops.Dropout(0.0, 1))
    assert torch.equal(Y0, Y1) and torch.equal(U0, U1)
    dX, dA, dB = ops.linear_bwd(d["q"], d["X"], d["dY"], d["A"], d["B"], 16.0, U=U0, drop=ops.Dropout(0.0, 1))
    D = np.ones((300, 448))
    bounds = adapter_bounds(d["Xr"], d["dYr"], d["Ar"], d["Br"], d["Wd"], 1.0, D, torch_to_f64(U0))
    for g, (ref, tol), name in zip((dX, dA, dB), bounds, ("dX", "dA", "dB")):
        within(g, ref, tol, name)


def test_nan_behind_the_mask_stays_out_of_u_and_da():
    M, N, K, r = 96, 128, 256, 8
    d = make(M, N, K, r, 7)
    keep = OD.keep_mask(M * K, 0.5, 13, 2).reshape(M, K)
    X = d["X"].clone()
    X[torch.from_numpy(~keep).cuda()] = float("nan")
    drop = ops.Dropout(0.5, 13, 2)
    _, U = ops.linear_fwd(d["q"], X, d["A"], d["B"], 16.0, save_u=True, drop=drop)
    _, U0 = ops.linear_fwd(d["q"], d["X"], d["A"], d["B"], 16.0, save_u=True, drop=drop)
    assert torch.equal(U, U0)
    a = ops.linear_bwd(d["q"], X, d["dY"], d["A"], d["B"], 16.0, U=U, drop=drop)
    b = ops.linear_bwd(d["q"], d["X"], d["dY"], d["A"], d["B"], 16.0, U=U, drop=drop)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_masks_of_two_offsets_differ_and_split_contraction():
    # 16448 columns of dY and few tiles: the contraction of dX is split
    M, N, K, r = 70, 16448, 256, 32
    d = make(M, N, K, r, 9)
    outs = []
    for off in (1, 2):
        drop = ops.Dropout(0.4, 5, off)
        D = OD.keep_mask(M * K, 0.4, 5, off).reshape(M, K) * OD.keep_scale(0.4)
        U = ops.linear_fwd(d["q"], d["X"], d["A"], d["B"], 16.0, save_u=True, drop=drop)[1]
        got = ops.linear_bwd(d["q"], d["X"], d["dY"], d["A"], d["B"], 16.0, U=U, drop=drop)
        bounds = adapter_bounds(d["Xr"], d["dYr"], d["Ar"], d["Br"], d["Wd"], 0.5, D, torch_to_f64(U))
        for g, (ref, tol), name in zip(got, bounds, ("dX", "dA", "dB")):
            within(g, ref, tol, name)
        outs.append(got[0])
    assert not torch.equal(outs[0], outs[1])


def test_refusals():
    d = make(64, 64, 64, 8, 10)
    X, A, B, q = d["X"], d["A"], d["B"], d["q"]
    for p in (-0.1, 1.0, 2.0, float("nan")):
        with pytest.raises(_lib.QloraError):
            ops.dropout(X, ops.Dropout(p, 1))
        with pytest.raises(_lib.QloraError):
            ops.linear_fwd(q, X, A, B, 16.0, drop=ops.Dropout(p, 1))
    with pytest.raises(_lib.QloraError):
        ops.linear_fwd(q, X, drop=ops.Dropout(0.1, 1))                      # no adapter
    with pytest.raises(_lib.QloraError):
        ops.linear_bwd(q, X, d["dY"], drop=ops.Dropout(0.1, 1))
    with pytest.raises(ValueError):
        ops.linear_bwd(q, X, d["dY"], A, B, 16.0, drop=ops.Dropout(0.1, 1), path="fused")
    with pytest.raises(ValueError):
        ops.linear_fwd(q, X, A, B, 16.0, drop=ops.Dropout(0.1, 1), path="fused")
    with pytest.raises(ValueError):
        ops.dropout(X.t(), ops.Dropout(0.1, 1))                              # strided
    with pytest.raises(ValueError):
        ops.dropout(X.float(), ops.Dropout(0.1, 1))
    with pytest.raises(ValueError):
        ops.dropout(X, ops.Dropout(0.1, 1, 0, torch.zeros(2, dtype=torch.int64, device="cuda")))
    with pytest.raises(ValueError):
        ops.dropout(X, ops.Dropout(0.1, 1, 0, torch.zeros(1, dtype=torch.int64)))
    with pytest.raises(_lib.QloraError):
        ops.linear_bwd(q, X, d["dY"], A, B, 16.0, drop=ops.Dropout(0.1, 1),
                       ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
