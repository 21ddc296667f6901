"""GPU: a split 8-bit product is the exact integer sum, as an unsplit one.

Rows whose largest magnitude is 127 have scale 1, so codes are the values. X
and the first half of W lie in [60, 127], so that every part of a split
contraction is far above 2^24, and the second half of W is minus the first but
for a few ones: the whole sum is a small integer, which parts rounded to fp32
would miss."""

import numpy as np
import pytest
import torch

from bit_quantized_finetuning_nf4_amd import ops
from tests.helpers import torch_to_f64
from tests.test_gpu_tiles import FEW, SIZES

pytestmark = pytest.mark.gpu

CASES = {n: (M, N, 128 * lines) for n, (M, N, lines) in SIZES.items() if "split" in n}
CASES.update({f"{M} tokens {N}x{K}": (M, N, K) for M, N, K in FEW if M >= 16 or N < 1024})
CASES["40 tokens 840x19840"] = (40, 840, 19840)


def to_gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).cuda()


def cancelling(rng, M, N, K):
    half = K // 2
    X = rng.integers(60, 128, (M, half)).astype(np.float64)
    X = np.concatenate([X, X], axis=1)
    X[:, 0] = X[:, half] = 127
    W = rng.integers(60, 127, (N, half)).astype(np.float64)
    W[:, 0] = 127
    V = -W
    cols = rng.integers(1, half, (N, 4))
    V[np.arange(N)[:, None], cols] += rng.choice([-1.0, 1.0], (N, 4))
    return X, np.concatenate([W, V], axis=1)


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("r", [0, 16, 40])
def test_the_sum_is_exact(name, r):
    M, N, K = CASES[name]
    print(f"[i8 split] {name} M{M} N{N} K{K} r{r}", flush=True)
    rng = np.random.default_rng(M + N + r)
    X, W = cancelling(rng, M, N, K)
    S = X @ W.T
    assert np.abs(S).max() <= 4 * 127 + 4 * 67 and np.abs(X).max() == 127
    w, xg = ops.i8_quantize(to_gpu(W)), to_gpu(X)
    assert (w.scale == 1).all()
    plain = ops.i8_matmul(ops.i8_quantize(xg), w)
    assert torch.equal(plain.cpu(), torch.from_numpy(S).to(torch.bfloat16))
    if r == 0:
        assert torch.equal(ops.i8_linear_fwd(w, xg), plain)
        return
    # alpha = r: s = 1.  A is sparse ones, B small integers: the adapter's term is an integer too, below 2^24 with the sum
    A = np.zeros((r, K))
    for j in range(r):
        A[j, rng.integers(0, K, 6)] = rng.choice([-1.0, 1.0], 6)
    B = rng.integers(-2, 3, (N, r)).astype(np.float64)
    want = S + X @ A.T @ B.T
    assert np.abs(want).max() < 2**24
    got = ops.i8_linear_fwd(w, xg, to_gpu(A), to_gpu(B), float(r))
    assert torch.equal(got.cpu(), torch.from_numpy(want).to(torch.bfloat16))


@pytest.mark.parametrize("name", CASES)
def test_same_bits_as_the_unsplit_product(name):
    M, N, K = CASES[name]
    print(f"[i8 split] {name} M{M} N{N} K{K}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    w = ops.i8_quantize(torch.randn((N, K), generator=gen, device="cuda").mul_(0.02).to(torch.bfloat16))
    X = torch.randn((M, K), generator=gen, device="cuda").to(torch.bfloat16)
    X[0] = 0
    if M > 2:
        X[2, 5] = float("inf")
    Y, want = ops.i8_linear_fwd(w, X), ops.i8_matmul(ops.i8_quantize(X), w)
    assert np.array_equal(torch_to_f64(Y), torch_to_f64(want), equal_nan=True)


def test_split_products_captured_and_on_two_streams():
    """Replays of a captured split product with eager calls between them, and two at once."""
    rng = np.random.default_rng(5)
    cases = []
    for M, N, K, r in ((40, 840, 19840, 16), (65, 9280, 5760, 64), (195, 8512, 9088, 128)):
        w = ops.i8_quantize(torch.randn((N, K), device="cuda").mul_(0.02).to(torch.bfloat16))
        X, A, B = (to_gpu(rng.standard_normal(s)) for s in ((M, K), (r, K), (N, r)))
        cases.append((w, X, A, B))
    call = lambda c, **kw: ops.i8_linear_fwd(*c, 16.0, **kw)
    want = [call(c) for c in cases]
    torch.cuda.synchronize()
    stream, other = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [torch.empty_like(y) for y in want]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        for c, o in zip(cases, outs):
            call(c, out=o)
    for _ in range(4):
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        for c, o, y in zip(cases, outs, want):
            assert torch.equal(o, y) and torch.equal(call(c), y)
    for _ in range(4):
        with torch.cuda.stream(stream):
            a = [call(c) for c in cases]
        with torch.cuda.stream(other):
            b = [call(c) for c in reversed(cases)]
        torch.cuda.synchronize()
        for y, s, t in zip(want, a, reversed(b)):
            assert torch.equal(s, y) and torch.equal(t, y)
