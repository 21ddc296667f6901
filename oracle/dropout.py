"""Dropout from a counter-based generator (fp64 numpy oracle).

Philox-4x32 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy
as 1, 2, 3", SC 2011, section 3.3): a round multiplies words 0 and 2 of the
counter by two constants and swaps halves; the key grows by two Weyl
constants per round.  Python integers, element by element blocks vectorised
over uint64.
"""

import numpy as np

MULT = (0xD2511F53, 0xCD9E8D57)
WEYL = (0x9E3779B9, 0xBB67AE85)
MASK32 = (1 << 32) - 1


def philox4x32(counters, key, rounds=7):
    """counters: uint32-valued array [n, 4]; key: two words.  Returns uint32 [n, 4]."""
    x = np.asarray(counters, dtype=np.uint64).reshape(-1, 4).copy()
    k = [int(key[0]), int(key[1])]
    for _ in range(rounds):
        p0, p1 = x[:, 0] * np.uint64(MULT[0]), x[:, 2] * np.uint64(MULT[1])
        hi0, lo0 = p0 >> np.uint64(32), p0 & np.uint64(MASK32)
        hi1, lo1 = p1 >> np.uint64(32), p1 & np.uint64(MASK32)
        x = np.stack([hi1 ^ x[:, 1] ^ np.uint64(k[0]), lo1, hi0 ^ x[:, 3] ^ np.uint64(k[1]), lo0], axis=1)
        k = [(k[0] + WEYL[0]) & MASK32, (k[1] + WEYL[1]) & MASK32]
    return x.astype(np.uint32)


def threshold(p):
    """Dropped halves out of 65536."""
    return min(65535, int(np.floor(65536.0 * p + 0.5)))


def keep_scale(p):
    return 65536.0 / (65536 - threshold(p))


def keep_mask(n, p, seed, offset=0, first=0):
    """Booleans: element first + i of the flattened tensor is kept."""
    lo, hi = first // 8, (first + n + 7) // 8
    blocks = np.arange(lo, hi, dtype=np.uint64)
    ctr = np.stack([blocks & np.uint64(MASK32), blocks >> np.uint64(32),
                    np.full_like(blocks, offset & MASK32), np.full_like(blocks, offset >> 32 & MASK32)], axis=1)
    words = philox4x32(ctr, (seed & MASK32, seed >> 32 & MASK32))
    halves = np.ascontiguousarray(words).view(np.uint16).reshape(-1).astype(np.int64)
    signed = np.where(halves >= 32768, halves - 65536, halves)
    return (signed >= threshold(p) - 32768)[first - 8 * lo:first - 8 * lo + n]


def drop(x, p, seed, offset=0):
    """drop(x) in fp64; dropped elements are 0 whatever they held."""
    x = np.asarray(x, dtype=np.float64)
    keep = keep_mask(x.size, p, seed, offset).reshape(x.shape)
    return np.where(keep, x * keep_scale(p), 0.0)


def linear_fwd_drop(Wd, X, A, B, alpha, p, seed, offset=0):
    """(Y, U): Y = X Wd^T + (alpha/r) U B^T, U = drop(X) A^T."""
    U = drop(X, p, seed, offset) @ A.T
    return X @ Wd.T + (alpha / A.shape[0]) * (U @ B.T), U


def linear_bwd_drop(Wd, X, dY, A, B, alpha, p, seed, offset=0, U=None):
    """(dX, dA, dB) of linear_fwd_drop."""
    s = alpha / A.shape[0]
    if U is None:
        U = drop(X, p, seed, offset) @ A.T
    G = dY @ B
    return dY @ Wd + s * drop(G @ A, p, seed, offset), s * (G.T @ drop(X, p, seed, offset)), s * (dY.T @ U)
