"""The gated feed-forward block and the adapters of many requests, in fp64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Reading R22 (the pages' models are LLaMA ones, whose feed-forward block joins
its gate and up linears by silu(G) * P; the pages do not spell it out):

    H = act(G) * P,  G and P the layers of "linear.py" on one X with the
    adapters stacked as in "group.py";
    dG = dH * P * act'(G) and dP = dH * act(G), rounded to fp32 and from there
    to bf16, are the gradients of the two layers' outputs.

Reading R23 (adapters of many requests): token m is the layer of "linear.py"
with the adapter of its own slot, s = scale[slot]; an id that is no slot has
none.  The slot's rank counts up to the next multiple of eight.
"""

import math

import numpy as np

from .bf16 import bf16_bits_to_f64, f32_to_bf16_bits
from .group import group_bwd, group_fwd


def act(x, name):
    """act(x) and act'(x)."""
    x = np.asarray(x, dtype=np.float64)
    # (1 + tanh z) / 2 = 1 / (1 + exp(-2 z)), which keeps its digits where tanh z is next to -1
    p, dp = x, 1.0
    if name != "silu":
        c = 2.0 * math.sqrt(2.0 / math.pi)
        p, dp = c * (x + 0.044715 * x**3), c * (1.0 + 3 * 0.044715 * x * x)
    with np.errstate(over="ignore"):
        s, rest = 1.0 / (1.0 + np.exp(-p)), 1.0 / (1.0 + np.exp(p))
    return x * s, s + x * s * rest * dp


def gated_fwd(Wds, X, A, B, alpha, name):
    """(H [M x F], [G | P] [M x 2 F])."""
    GU = group_fwd(Wds, X, A, B, alpha)
    F = GU.shape[1] // 2
    return act(GU[:, :F], name)[0] * GU[:, F:], GU


def gated_dy(dH, GU, name):
    """[dG | dP], rounded to fp32 and then to bf16."""
    F = dH.shape[1]
    a, slope = act(GU[:, :F], name)
    dY = np.concatenate((dH * GU[:, F:] * slope, dH * a), axis=1)
    return bf16_bits_to_f64(f32_to_bf16_bits(dY.astype(np.float32))).reshape(dY.shape)


def gated_bwd(Wds, X, dH, GU, A, B, alpha, name):
    """(dX, dA, dB), U computed again."""
    return group_bwd(Wds, X, gated_dy(dH, GU, name), A, B, alpha)


def many_fwd(Wd, X, A, B, scale, ids, rank=None):
    """Y [M x N]; A [S x R x K], B [S x N x R]."""
    S, R = A.shape[0], A.shape[1]
    Y = X @ Wd.T
    for m, a in enumerate(ids):
        if 0 <= a < S:
            r = R if rank is None else min(R, -(-max(0, int(rank[a])) // 8) * 8)
            Y[m] += scale[a] * (B[a][:, :r] @ (A[a][:r] @ X[m]))
    return Y
