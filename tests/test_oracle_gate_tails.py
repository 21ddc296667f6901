"""The oracle's activations and slopes far from zero, against decimal arithmetic of 60 digits."""

from decimal import Decimal, getcontext

import numpy as np
import pytest

import oracle

getcontext().prec = 60
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494")


def exact(x, name):
    """act(x) = x sigma(p(x)) and its slope, to about 50 digits."""
    x = Decimal(x)
    a = Decimal(0.044715)   # the double nearest, as every program has it
    c = 2 * (2 / PI).sqrt()
    p, dp = (x, Decimal(1)) if name == "silu" else (c * (x + a * x**3), c * (1 + 3 * a * x * x))
    s, r = 1 / (1 + (-p).exp()), 1 / (1 + p.exp())
    return x * s, s + x * s * r * dp


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_tails(name):
    # 2^-50 of the value: a dozen roundings, and the exponent's argument, rounded by 3 2^-53 |p|, moves exp by as much
    for x in np.concatenate((np.linspace(-9, 9, 181), [-40.0, -20.0, 20.0, 40.0] if name == "silu" else [12.0, 30.0])):
        p = abs(x) if name == "silu" else 1.6 * abs(x + 0.044715 * x**3)
        got = oracle.act(np.array([x]), name)
        want = exact(float(x), name)
        # the slope is a difference of two terms near its zero
        size = (abs(float(want[0])), abs(float(want[1])) + abs(float(want[0])) * (1 if name == "silu" else 1.6 + 0.22 * x * x))
        for g, w, n in zip(got, want, size):
            assert abs(Decimal(float(g[0])) - w) <= Decimal((2.0**-50 + 3 * 2.0**-53 * p) * n), (x, float(g[0]), float(w))
