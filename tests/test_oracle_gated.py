"""Pins of the gated block's and the many adapters' oracle (oracle/gated.py)
against formulations other than its own."""

import math

import numpy as np
import pytest

import oracle


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_activation_is_x_times_a_logistic_and_its_slope_a_difference(name):
    x = np.linspace(-30, 30, 6001)
    p = x if name == "silu" else 2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x**3)
    with np.errstate(over="ignore"):
        want = np.where(p >= 0, x / (1 + np.exp(-p)), x * np.exp(np.minimum(p, 0)) / (1 + np.exp(np.minimum(p, 0))))
    a, slope = oracle.act(x, name)
    np.testing.assert_allclose(a, want, rtol=1e-10, atol=1e-14)
    h = 1e-5
    diff = (oracle.act(x + h, name)[0] - oracle.act(x - h, name)[0]) / (2 * h)
    np.testing.assert_allclose(slope, diff, atol=1e-8)


def test_gelu_is_near_the_error_functions():
    x = np.linspace(-4, 4, 401)
    want = np.array([0.5 * v * (1 + math.erf(v / math.sqrt(2))) for v in x])
    assert np.abs(oracle.act(x, "gelu")[0] - want).max() < 1e-3


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_gradients_are_differences_of_the_loss(name):
    M, F, K, r, alpha = 3, 8, 16, 4, 8.0
    rng = np.random.default_rng(0)
    Ws = [rng.standard_normal((F, K)) * 0.3 for _ in range(2)]
    X, dH = rng.standard_normal((M, K)), rng.standard_normal((M, F))
    A, B = rng.standard_normal((2 * r, K)) * 0.3, rng.standard_normal((2 * F, r)) * 0.3
    GU = oracle.gated_fwd(Ws, X, A, B, alpha, name)[1]
    grads = oracle.gated_bwd(Ws, X, dH, GU, A, B, alpha, name)
    loss = lambda X, A, B: float((dH * oracle.gated_fwd(Ws, X, A, B, alpha, name)[0]).sum())
    args, h = [X, A, B], 1e-5
    for i, g in enumerate(grads):
        for _ in range(10):
            at = tuple(rng.integers(0, n) for n in args[i].shape)
            up, dn = [a.copy() for a in args], [a.copy() for a in args]
            up[i][at] += h
            dn[i][at] -= h
            # the oracle's dG and dP carry one rounding to bf16
            assert abs((loss(*up) - loss(*dn)) / (2 * h) - g[at]) <= 2.0**-8 * np.abs(g).max() + 1e-6


def test_rounding_in_between_is_to_bf16():
    rng = np.random.default_rng(1)
    dH, GU = rng.standard_normal((5, 8)), rng.standard_normal((5, 16))
    dY = oracle.gated_dy(dH, GU, "silu")
    assert np.array_equal(oracle.bf16_bits_to_f64(oracle.f32_to_bf16_bits(dY.astype(np.float32))).reshape(dY.shape), dY)
    s = 1 / (1 + np.exp(-GU[:, :8]))
    np.testing.assert_allclose(dY[:, 8:], dH * GU[:, :8] * s, rtol=2.0**-8)


def test_many_is_one_adapter_per_token():
    M, N, K, S, R = 9, 8, 16, 4, 16
    rng = np.random.default_rng(2)
    W, X = rng.standard_normal((N, K)), rng.standard_normal((M, K))
    A, B, scale = rng.standard_normal((S, R, K)), rng.standard_normal((S, N, R)), rng.standard_normal(S)
    ids = np.array([0, 3, 3, -1, 4, 1, 2, 0, 99])
    rank = np.array([16, 8, 0, 3])
    Y = oracle.many_fwd(W, X, A, B, scale, ids, rank)
    # the same as one product with a weight merged per token
    for m, a in enumerate(ids):
        Wm = W.copy()
        if 0 <= a < S:
            r = (16, 8, 0, 8)[a]
            Wm += scale[a] * np.einsum("nj,jk->nk", B[a][:, :r], A[a][:r])
        np.testing.assert_allclose(Y[m], Wm @ X[m], rtol=1e-12, atol=1e-12)
