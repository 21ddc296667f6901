"""Pins of the dropout and 8-bit oracles (CPU)."""

import numpy as np
import pytest

from oracle import dropout as D
from oracle import i8 as I


# Known answers of Philox-4x32 published with the generator's reference
# implementation: counter and key of all zeros and all ones, 7 and 10 rounds.
@pytest.mark.parametrize("rounds,word,want", [
    (7, 0x00000000, (0x5F6FB709, 0x0D893F64, 0x4F121F81, 0x4F730A48)),
    (7, 0xFFFFFFFF, (0x5207DDC2, 0x45165E59, 0x4D8EE751, 0x8C52F662)),
    (10, 0x00000000, (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    (10, 0xFFFFFFFF, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
])
def test_philox_known_answers(rounds, word, want):
    got = D.philox4x32([[word] * 4], (word, word), rounds)[0]
    assert tuple(int(v) for v in got) == want


@pytest.mark.parametrize("p", [0.0, 1e-6, 0.05, 0.1, 0.5, 0.9, 0.9999999])
def test_mask_rate_and_scale(p):
    n = 1 << 20
    keep = D.keep_mask(n, p, seed=5, offset=9)
    t = D.threshold(p)
    q = 1 - t / 65536
    # binomial: five standard deviations
    assert abs(keep.mean() - q) <= 5 * np.sqrt(q * (1 - q) / n) + 1e-12
    assert D.keep_scale(p) == pytest.approx(1 / q)
    if t == 0:
        assert keep.all()


def test_mask_depends_on_seed_offset_and_position_only():
    a = D.keep_mask(4096, 0.5, seed=1, offset=2)
    assert np.array_equal(a, D.keep_mask(4096, 0.5, seed=1, offset=2))
    assert np.array_equal(a[1234:1300], D.keep_mask(66, 0.5, 1, 2, first=1234))
    for other in (D.keep_mask(4096, 0.5, 2, 2), D.keep_mask(4096, 0.5, 1, 3), D.keep_mask(4096, 0.5, 1 << 32, 2),
                  D.keep_mask(4096, 0.5, 1, 2 + (1 << 32))):
        # independent fair bits agree half the time, five standard deviations
        assert abs((a == other).mean() - 0.5) <= 5 * 0.5 / np.sqrt(4096)


def test_dropped_linear_gradients_match_differences():
    rng = np.random.default_rng(3)
    M, N, K, r, alpha = 5, 16, 24, 8, 16.0
    W, X, A, B, dY = (rng.standard_normal(s) for s in ((N, K), (M, K), (r, K), (N, r), (M, N)))
    arg = (alpha, 0.3, 77, 5)
    f = lambda X, A, B: (D.linear_fwd_drop(W, X, A, B, *arg)[0] * dY).sum()
    dX, dA, dB = D.linear_bwd_drop(W, X, dY, A, B, *arg)
    for g, pos, args in ((dX, 0, (X, A, B)), (dA, 1, (X, A, B)), (dB, 2, (X, A, B))):
        for _ in range(5):
            step = rng.standard_normal(g.shape)
            lo, hi = list(args), list(args)
            lo[pos], hi[pos] = args[pos] - step, args[pos] + step
            # f is linear in each argument: central differences are exact up to fp64 rounding
            assert (f(*hi) - f(*lo)) / 2 == pytest.approx((g * step).sum(), rel=1e-9)


def test_i8_quantize():
    x = np.array([[0.0, 0.0, 0.0, 0.0], [1.0, -1.0, 0.5, -0.5], [127.0, 0.5, 1.5, -2.5], [np.inf, 1.0, 2.0, 3.0],
                  [np.nan, 1.0, 2.0, 3.0], [2.0**-133, -2.0**-133, 0.0, 0.0], [3e38, 1e38, 0.0, -3e38]])
    q, s = I.i8_quantize(x)
    assert q.tolist() == [[0, 0, 0, 0], [127, -127, 64, -64], [127, 0, 2, -2], [0, 0, 0, 0], [0, 0, 0, 0],
                          [127, -127, 0, 0], [127, 42, 0, -127]]
    assert s[0] == 0 and np.isnan(s[3]) and np.isnan(s[4]) and s[1] == np.float32(1 / 127)


def test_i8_round_trip_is_within_half_a_step():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((32, 200))
    q, s = I.i8_quantize(x)
    assert (np.abs(q * s[:, None].astype(np.float64) - x) <= 0.5001 * s[:, None]).all()
