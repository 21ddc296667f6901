"""The gated block's gradients against differences of its loss, sum(dH o H).

A gradient g is read along a direction in which every element adds to the
result: sign(g) on the elements that their error's bound leaves known best, so
that the sum of the errors stays far below the sum itself.  dH is zero but for
three tokens and the sixteen features whose gates are largest there: every sum behind g has few terms, whatever
the shape, and its bound is of g's own size.

The bound, element by element: GU is rounded by E = 2^-8 of its value, which
moves dG = dH P act'(G) by |dH| E (|P act'| + max |act''| |G P|) and dP = dH
act(G) by |dH| max |act'| E |G|; both are rounded by E once more, U by E, dX by
E.  1.05 covers the products of these and fp32's sums.  max |act'| is 1.2, max
|act''| 0.5 (silu) or 0.8 (gelu: sqrt(2 / pi) at 0).

The CPU tests plant mistakes in the gradients of the definition and see that
each is further off than the bound allows.
"""

import math

import numpy as np
import pytest
import torch

import oracle
from bit_quantized_finetuning_nf4_amd import ops, synth
from tests.helpers import bits_to_torch, torch_to_f64

E = 2.0**-8
ALPHA = 16.0
STEP = 2.0**-4   # of an element's mean size: a straight line to 5e-4 of the difference

# tokens x features x K, rank: streamed, dequantized in small tiles, in 256-token tiles
SHAPES = [(3, 72, 64, 8), (17, 104, 128, 16), (70, 264, 192, 8), (330, 136, 128, 16), (1040, 4104, 64, 8)]


def to_bf16(a):
    """(bit patterns, their values)."""
    bits = synth.to_bf16_bits(a)
    return bits, oracle.bf16_bits_to_f64(bits).reshape(np.shape(a))


class Case:
    """Inputs of one call, as bits or codes and as fp64 values."""

    def __init__(self, M, N, K, r, name):
        rng = np.random.default_rng(M + r)
        self.name, self.codes, self.Ws = name, [], []
        for _ in range(2):
            blocks = N * K // 64
            w = (rng.integers(0, 256, N * K // 2, dtype=np.uint8), rng.integers(128, 256, blocks, dtype=np.uint8),
                 (rng.random(-(-blocks // 256)) * 0.3 + 0.3).astype(np.float32))
            self.codes.append((N, K) + w)
            self.Ws.append(oracle.bf16_bits_to_f64(oracle.dequant(*w, N * K)).reshape(N, K))
        made = [to_bf16(rng.standard_normal(shape) * std)
                for shape, std in (((M, K), 4 / math.sqrt(K)), ((2 * r, K), 0.15), ((2 * N, r), 0.15))]
        self.X, self.A, self.B = (m[1] for m in made)
        self.s = oracle.lora_scale(ALPHA, r)
        self.GU = oracle.gated_fwd(self.Ws, self.X, self.A, self.B, ALPHA, name)[1]
        tokens = rng.choice(M, 3, replace=False)
        # (act's second term changes its sign with the gate)
        features = np.argsort(self.GU[tokens, :N].min(axis=0))[-16:]
        dH = np.zeros((M, N))
        dH[np.ix_(tokens, features)] = rng.standard_normal((3, 16))
        made.append(to_bf16(dH))
        self.bits, self.dH = [m[0] for m in made], made[3][1]

    def pairs(self):
        """(W, A, B, U) of gate and of up."""
        return [(W, A, B, self.X @ A.T) for W, A, B in zip(self.Ws, np.split(self.A, 2), np.split(self.B, 2))]

    def grads(self, mistake=None):
        """dX, dA, dB with nothing rounded in between."""
        G, P = np.split(self.GU, 2, axis=1)
        a, slope = oracle.act(G, self.name)
        if mistake == "slope":   # act' without its second term
            slope = np.where(G == 0, 0.5, a / np.where(G == 0, 1.0, G))
        dY = [self.dH * P * slope, self.dH * a]
        if mistake == "no dP":
            dY[1] = 0 * dY[1]
        if mistake == "exchanged":
            dY.reverse()
        dX, dA, dB = 0.0, [], []
        for d, (W, A, B, U) in zip(dY, self.pairs()):
            T = self.s * (d @ B)
            dX = dX + d @ W + (0 if mistake == "no adapter" else T @ A)
            dA.append(T.T @ self.X)
            dB.append(self.s * (d.T @ U))
        out = [dX, np.concatenate(dA), np.concatenate(dB)]
        return [0.5 * g for g in out] if mistake == "halved" else out

    def bounds(self):
        """What the kernels' dX, dA, dB may be off."""
        G, P = np.split(np.abs(self.GU), 2, axis=1)
        a, slope = (np.abs(v) for v in oracle.act(self.GU[:, :G.shape[1]], self.name))
        h, bend = np.abs(self.dH), 0.5 if self.name == "silu" else 0.8
        err = [h * E * (2 * P * slope + bend * G * P), h * E * (1.2 * G + a)]
        bX, bA, bB = E * np.abs(self.grads()[0]), [], []
        for e, d, (W, A, B, U) in zip(err, [h * P * slope, h * a], self.pairs()):
            t = self.s * (e @ np.abs(B))
            bX = bX + e @ np.abs(W) + t @ np.abs(A)
            bA.append(t.T @ np.abs(self.X))
            bB.append(self.s * ((e + E * d).T @ np.abs(U)))
        return [1.05 * b for b in (bX, np.concatenate(bA), np.concatenate(bB))]

    def lines(self):
        """For X, A and B: (bits of the direction's two ends, their difference, the loss's, what the gradient summed
        along it may be off, what the loss of rounded outputs may)."""
        out = []
        for i, (g, bound) in enumerate(zip(self.grads(), self.bounds())):
            known = np.abs(g) / np.maximum(bound, 1e-300)
            args = [self.X, self.A, self.B]
            base = args[i]
            move = np.sign(g) * (known >= min(16.0, np.quantile(known[g != 0], 0.9))) * np.abs(base).mean() * STEP
            ends = [to_bf16(base + sign * move) for sign in (1, -1)]
            delta, loss, rounding = ends[0][1] - ends[1][1], [], 0.0
            for _, v in ends:
                args[i] = v
                H = oracle.gated_fwd(self.Ws, *args, ALPHA, self.name)[0]
                loss.append(float((self.dH * H).sum()))
                rounding += 1.05 * E * float(np.abs(self.dH * H).sum())
            line = loss[0] - loss[1]
            slack = float((bound * np.abs(delta)).sum()) + abs(line - float((g * delta).sum()))
            out.append(([e[0] for e in ends], delta, line, slack, rounding))
        return out


@pytest.mark.parametrize("name", ["silu", "gelu"])
@pytest.mark.parametrize("shape", SHAPES)
def test_a_mistake_is_further_off_than_the_bound(shape, name):
    case = Case(*shape, name)
    lines = case.lines()
    for g, (_, delta, line, slack, rounding) in zip(case.grads(), lines):
        assert abs(float((g * delta).sum()) - line) <= slack < 0.1 * line and rounding < 0.25 * line
    for mistake in ("halved", "slope", "no dP", "exchanged", "no adapter"):
        for i, g in enumerate(case.grads(mistake)):
            _, delta, line, slack, _ = lines[i]
            if mistake != "no adapter" or i == 0:
                assert abs(float((g * delta).sum()) - line) > slack, (mistake, "XAB"[i])


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["silu", "gelu"])
@pytest.mark.parametrize("shape", SHAPES)
def test_gradients_are_differences_of_the_loss(shape, name):
    print(f"[differences] {shape} {name}", flush=True)
    case = Case(*shape, name)
    qs = [ops.QuantizedWeight(N, K, *(torch.from_numpy(a.copy()).cuda() for a in w)) for N, K, *w in case.codes]
    X, A, B, dH = (bits_to_torch(b) for b in case.bits)
    _, GU, U = ops.gated_fwd(qs, X, A, B, ALPHA, act=name, save=True)
    grads = ops.gated_bwd(qs, X, dH, GU, A, B, ALPHA, act=name, U=U)
    for i, (ends, delta, line, slack, rounding) in enumerate(case.lines()):
        along = float((torch_to_f64(grads[i]) * delta).sum())
        assert abs(along - line) <= slack, ("XAB"[i], along, line, slack)
        loss = []
        for bits in ends:
            args = [X, A, B]
            args[i] = bits_to_torch(bits).view(args[i].shape)
            loss.append(float((case.dH * torch_to_f64(ops.gated_fwd(qs, *args, ALPHA, act=name))).sum()))
        assert abs(loss[0] - loss[1] - line) <= rounding, ("XAB"[i], loss, line, rounding)
        assert abs(loss[0] - loss[1] - along) <= slack + rounding
