"""Timed cases of the adapter-dropout and 8-bit linear operators.

Kinds of case:

  dropout   y = drop(x), elementwise on bf16 (its gradient is the same map
            applied to dy)
  nf4_fwd   a frozen NF4 linear with its LoRA adapter under dropout, forward:
            Y = X deq(W)^T + s U B^T with U = drop(X) A^T; returns Y and U
  nf4_bwd   its backward: dX = dY deq(W) + s drop'(dY B A),
            dA = s (dY B)^T drop(X), dB = s dY^T U
  i8_quant  bf16 rows -> 8-bit integers and one scale per row
  i8_fwd    the linear with an 8-bit frozen weight (one scale per output
            channel) and 8-bit inputs (one scale per token), with its adapter
  i8_bwd    the backward of that linear; the gradient stays in 16 bits

Dropout masks come from Philox-4x32 with 7 rounds (Salmon, Moraes, Dror and
Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011): element i of
the row-major tensor takes 16-bit half i % 8 of the block whose counter is
i // 8 (low 64 bits) and the offset (high 64 bits), under the seed as key; it
is kept where the half, as a signed number, is at least round(65536 p) -
32768, and kept values are divided by the share that is kept.

With `own` false, run() uses elementary torch operations in 32 bits (64 where
a value is to be rounded to an integer); with `own` true it calls
bit_quantized_finetuning_nf4_amd.ops.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
M32 = 0xFFFFFFFF

NF4_BITS = (0xBF800000, 0xBF3239B1, 0xBF066B2E, 0xBECA329E, 0xBE91A24B, 0xBE3D353D, 0xBDBA7869, 0x00000000,
            0x3DA2FB01, 0x3E24CADF, 0x3E7C04DA, 0x3EAD0336, 0x3EE1A4B5, 0x3F1007A9, 0x3F3913B0, 0x3F800000)


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one token's hidden state of the 7B layer set: the smallest call, all latency
        dict(name="dropout_token", kind="dropout", M=1, K=4096, p=0.1),
        # the down projection's input in the 65B layer set: a pure stream
        dict(name="dropout_65b", kind="dropout", M=4096, K=22016, p=0.05),
        # the single small linear (rank 8)
        dict(name="nf4_fwd_small", kind="nf4_fwd", M=256, N=1024, K=1024, r=8, p=0.1),
        # the 13B layer set's gate projection in training
        dict(name="nf4_fwd_13b_gate", kind="nf4_fwd", M=2048, N=13824, K=5120, r=64, p=0.05),
        # the 7B layer set's query projection, backward: the shortest contraction under the mask
        dict(name="nf4_bwd_7b_q", kind="nf4_bwd", M=2048, N=4096, K=4096, r=64, p=0.1),
        # the 65B layer set's down projection, backward: the largest training call
        dict(name="nf4_bwd_65b_down", kind="nf4_bwd", M=4096, N=8192, K=22016, r=64, p=0.05),
        # quantizing the 65B layer set's gate weight once at load
        dict(name="i8_quant_65b_gate", kind="i8_quant", M=22016, K=8192),
        # serving, one token through the 65B query projection and its adapter
        dict(name="i8_fwd_token", kind="i8_fwd", M=1, N=8192, K=8192, r=64, p=0.0),
        # serving, a batch of sixteen through the 65B gate projection, without an adapter
        dict(name="i8_fwd_batch16", kind="i8_fwd", M=16, N=22016, K=8192, r=0, p=0.0),
        # a ragged prompt through the 7B gate projection, rank 16
        dict(name="i8_fwd_ragged", kind="i8_fwd", M=333, N=11008, K=4096, r=16, p=0.0),
        # the 65B gate projection in training, adapter under dropout
        dict(name="i8_fwd_65b_gate", kind="i8_fwd", M=4096, N=22016, K=8192, r=64, p=0.05),
        # the 13B down projection in training, backward
        dict(name="i8_bwd_13b_down", kind="i8_bwd", M=2048, N=5120, K=13824, r=64, p=0.05),
    ]


def _spread(rng, lo, hi, step):
    """A multiple of `step` between lo and hi, even over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    kind = rng.choice(("dropout", "nf4_fwd", "nf4_bwd", "i8_quant", "i8_fwd", "i8_fwd", "i8_bwd"))
    if kind == "dropout":
        return dict(kind=kind, M=_spread(rng, 1, 4096, 1), K=_spread(rng, 8, 22016, 1), p=round(rng.uniform(0.01, 0.6), 3))
    if kind == "i8_quant":
        return dict(kind=kind, M=_spread(rng, 1, 22016, 1), K=_spread(rng, 64, 8192, 8))
    step = 64 if kind.startswith("nf4") else 8
    while True:
        M = _spread(rng, 1 if kind == "i8_fwd" else 64, 4096, 1)
        N, K = _spread(rng, 512, 22016, step), _spread(rng, 512, 22016, step)
        if M * N * K <= 4096 * 8192 * 22016:
            break
    r = rng.choice((8, 16, 32, 64, 128)) if kind != "i8_fwd" else rng.choice((0, 8, 16, 32, 64, 128))
    p = 0.0 if r == 0 or (kind.startswith("i8") and rng.random() < 0.4) else round(rng.uniform(0.01, 0.5), 3)
    return dict(kind=kind, M=M, N=N, K=K, r=r, p=p)


def work(case):
    k, M, K = case["kind"], case["M"], case["K"]
    if k == "dropout":
        return {"bytes": 4 * M * K, "flops": M * K}
    if k == "i8_quant":
        return {"bytes": 3 * M * K + 4 * M, "flops": 2 * M * K}
    N, r = case["N"], case["r"]
    wb = N * K / 2 + N * K / 64 + N * K / 4096 if k.startswith("nf4") else N * K + 4 * N
    adapter = 2 * r * (N + K)
    if k.endswith("fwd"):
        u = 2 * M * r if r else 0
        return {"bytes": int(2 * M * K + wb + adapter + 2 * M * N + u), "flops": 2 * M * N * K + 2 * M * r * (N + K)}
    return {"bytes": int(2 * M * K + 2 * M * N + 2 * M * r + wb + adapter + 2 * M * K + 4 * r * (N + K)),
            "flops": 2 * M * N * K + 4 * M * r * (N + K)}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

ALPHA = 16.0


def _normal(gen, shape, std, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).mul_(std).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    k, M, K = case["kind"], case["M"], case["K"]
    st = {"case": case, "seed": 7 + 1000003 * seed, "offset": 12 + seed}
    if k in ("dropout", "i8_quant"):
        st["x"] = _normal(gen, (M, K), 1.0 if k == "dropout" else 0.02)
        return st
    N, r = case["N"], case["r"]
    st["X"] = _normal(gen, (M, K), 1.0)
    if k.startswith("nf4"):
        # uniform codes (the levels are normal quantiles), block constants spread below their group's largest
        blocks = N * K // 64
        st["codes"] = torch.randint(0, 256, (N * K // 2,), generator=gen, device=DEV, dtype=torch.uint8)
        st["absmax_q"] = (torch.randn(blocks, generator=gen, device=DEV) * 25 + 160).clamp_(80, 255).to(torch.uint8)
        st["group_scale"] = torch.rand((blocks + 255) // 256, generator=gen, device=DEV) * 0.02 + 0.07
    else:
        # rows padded with zeros to whole 128-byte lines
        W = torch.randn((N, K), generator=gen, device=DEV) * 0.02
        st["w_scale"] = W.abs().amax(1) / 127
        st["w_codes"] = torch.zeros((N, (K + 127) // 128 * 128), device=DEV, dtype=torch.int8)
        st["w_codes"][:, :K] = torch.round(W / st["w_scale"][:, None]).to(torch.int8)
    st["A"] = _normal(gen, (r, K), 0.01) if r else None
    st["B"] = _normal(gen, (N, r), 0.01) if r else None
    if k.endswith("bwd"):
        st["dY"] = _normal(gen, (M, N), 1.0)
        st["U"] = _normal(gen, (M, r), 0.01 * math.sqrt(K))
    return st


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------

def _halves(n, seed, offset, device):
    """The signed 16-bit halves of elements 0..n-1, int64."""
    c0 = torch.arange((n + 7) // 8, device=device, dtype=torch.int64)
    c1 = c0 >> 32
    c0 = c0 & M32
    c2 = torch.full_like(c0, offset & M32)
    c3 = torch.full_like(c0, offset >> 32 & M32)
    k0, k1 = seed & M32, seed >> 32 & M32
    for _ in range(7):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57     # 64-bit products, modulo 2^64
        c0, c1, c2, c3 = (b >> 32 & M32) ^ c1 ^ k0, b & M32, (a >> 32 & M32) ^ c3 ^ k1, a & M32
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    w = torch.stack((c0, c1, c2, c3), -1)
    h = torch.stack((w & 0xFFFF, w >> 16), -1).reshape(-1)[:n]
    return torch.where(h >= 32768, h - 65536, h)


def _threshold(p):
    return min(65535, int(math.floor(65536.0 * p + 0.5)))


def _dropped(x, p, seed, offset):
    """drop(x) in 32 bits."""
    if p == 0.0:
        return x.float()
    t = _threshold(p)
    keep = _halves(x.numel(), seed, offset, x.device).view(x.shape) >= t - 32768
    return torch.where(keep, x.float() * (65536.0 / (65536 - t)), torch.zeros((), device=x.device))


def _nf4_weight(st):
    c = st["case"]
    levels = torch.from_numpy(np.array(NF4_BITS, dtype=np.uint32).view(np.float32)).to(DEV)
    codes = torch.stack((st["codes"] & 15, st["codes"] >> 4), -1).reshape(-1, 64).long()
    q8 = (torch.arange(256, device=DEV, dtype=torch.float64) / 255).float()
    groups = torch.arange(st["absmax_q"].numel(), device=DEV) // 256
    t = q8[st["absmax_q"].long()] * st["group_scale"][groups]
    return (levels[codes] * t[:, None]).to(torch.bfloat16).float().view(c["N"], c["K"])


def _quant(x):
    """Whole numbers in [-127, 127] (float64) and the scale of each row."""
    amax = x.double().abs().amax(1, keepdim=True)
    q = torch.round(127.0 * x.double() / torch.where(amax > 0, amax, torch.ones_like(amax)))
    return q, (amax / 127.0).float()


def _plain(st):
    c = st["case"]
    k, p, K = c["kind"], c.get("p", 0.0), c["K"]
    if k == "dropout":
        return _dropped(st["x"], p, st["seed"], st["offset"]).to(torch.bfloat16)
    if k == "i8_quant":
        q, scale = _quant(st["x"])
        return {"q": q.to(torch.int8), "scale": scale.view(-1)}
    s = ALPHA / c["r"] if c["r"] else 0.0
    X = st["X"]
    if k.endswith("fwd"):
        if k == "nf4_fwd":
            Y = X.float() @ _nf4_weight(st).t()
        else:
            q, sx = _quant(X)
            Y = (q.float() @ st["w_codes"][:, :K].float().t()) * (sx * st["w_scale"])
        if not c["r"]:
            return {"Y": Y.to(torch.bfloat16)}
        U = _dropped(X, p, st["seed"], st["offset"]) @ st["A"].float().t()
        return {"Y": (Y + s * (U @ st["B"].float().t())).to(torch.bfloat16), "U": U.to(torch.bfloat16)}
    dY = st["dY"].float()
    W = _nf4_weight(st) if k == "nf4_bwd" else (st["w_codes"][:, :K].float() * st["w_scale"][:, None]).to(torch.bfloat16).float()
    A, B = st["A"].float(), st["B"].float()
    G = dY @ B
    dX = dY @ W + _dropped(s * (G @ A), p, st["seed"], st["offset"])
    dA = s * (G.t() @ _dropped(X, p, st["seed"], st["offset"]))
    dB = s * (dY.t() @ st["U"].float())
    return {"dX": dX.to(torch.bfloat16), "dA": dA, "dB": dB}


# --------------------------------------------------------------------------
# the framework's operators
# --------------------------------------------------------------------------

def _framework(st):
    from bit_quantized_finetuning_nf4_amd import ops

    c = st["case"]
    k = c["kind"]
    drop = ops.Dropout(c["p"], st["seed"], st["offset"]) if c.get("p", 0.0) > 0.0 else None
    if k == "dropout":
        return ops.dropout(st["x"], drop)
    if k == "i8_quant":
        w = ops.i8_quantize(st["x"])
        return {"q": w.codes[:, :c["K"]], "scale": w.scale}
    if k.startswith("nf4"):
        w = ops.QuantizedWeight(c["N"], c["K"], st["codes"], st["absmax_q"], st["group_scale"])
        fwd, bwd = ops.linear_fwd, ops.linear_bwd
    else:
        w = ops.Int8Weight(c["N"], c["K"], st["w_codes"], st["w_scale"])
        fwd, bwd = ops.i8_linear_fwd, ops.i8_linear_bwd
    if k.endswith("fwd"):
        if not c["r"]:
            return {"Y": fwd(w, st["X"])}
        Y, U = fwd(w, st["X"], st["A"], st["B"], ALPHA, save_u=True, drop=drop)
        return {"Y": Y, "U": U}
    dX, dA, dB = bwd(w, st["X"], st["dY"], st["A"], st["B"], ALPHA, U=st["U"], drop=drop)
    return {"dX": dX, "dA": dA, "dB": dB}


def run(state):
    if own:
        return _framework(state)
    return _plain(state)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _keep64(shape, p, seed, offset):
    """The kept share of each element: 0 or 1 / (1 - p'), p' the probability in 1/65536 (numpy, unsigned)."""
    t = _threshold(p)
    if p == 0.0:
        return torch.ones(shape, device=DEV, dtype=torch.float64)
    n = int(np.prod(shape))
    lo, shift = np.uint64(M32), np.uint64(32)
    ctr = np.arange(-(-n // 8), dtype=np.uint64)
    x = [ctr & lo, ctr >> shift, np.full_like(ctr, offset & M32), np.full_like(ctr, (offset >> 32) & M32)]
    key = [seed & M32, (seed >> 32) & M32]
    for _ in range(7):
        first, second = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(second >> shift) ^ x[1] ^ np.uint64(key[0]), second & lo,
             (first >> shift) ^ x[3] ^ np.uint64(key[1]), first & lo]
        key = [(key[0] + 0x9E3779B9) % 2**32, (key[1] + 0xBB67AE85) % 2**32]
    words = np.stack([v.astype(np.uint32) for v in x], 1)
    halves = np.ascontiguousarray(words).view("<i2").reshape(-1)[:n].reshape(shape)
    return torch.from_numpy(halves >= t - 32768).to(DEV).double() / (1.0 - t / 65536.0)


def _nf4_weight64(st):
    c = st["case"]
    out = torch.empty(c["N"] * c["K"], device=DEV, dtype=torch.float64)
    levels = torch.from_numpy(np.array(NF4_BITS, dtype=np.uint32).view(np.float32).astype(np.float64)).to(DEV)
    # a stored value is the fp32 product of fp32 numbers, rounded to bf16: products of two 24-bit numbers are exact in 64 bits
    scale = (st["absmax_q"].double() / 255).float().double() * st["group_scale"].double().repeat_interleave(256)[:st["absmax_q"].numel()]
    scale = scale.float().double().repeat_interleave(32)
    out[0::2] = (levels[(st["codes"] % 16).int()] * scale).float().bfloat16().double()
    out[1::2] = (levels[(st["codes"] // 16).int()] * scale).float().bfloat16().double()
    return out.view(c["N"], c["K"])


def exact(case, seed):
    st = prepare(case, seed)
    k, p, K = case["kind"], case.get("p", 0.0), case["K"]
    if k == "dropout":
        return st["x"].double() * _keep64(tuple(st["x"].shape), p, st["seed"], st["offset"])
    if k == "i8_quant":
        top = torch.linalg.vector_norm(st["x"].double(), math.inf, dim=1)
        return {"q": (st["x"].double() * 127 / top.clamp_min(1e-300)[:, None]).round().to(torch.int8), "scale": top / 127}
    s = ALPHA / case["r"] if case["r"] else 0.0
    X = st["X"].double()
    D = _keep64(tuple(X.shape), p, st["seed"], st["offset"]) if case["r"] else None
    if k.endswith("fwd"):
        if k == "nf4_fwd":
            Y = torch.matmul(X, _nf4_weight64(st).T)
        else:
            top = torch.linalg.vector_norm(X, math.inf, dim=1)[:, None]
            ints = (X * 127 / top.clamp_min(1e-300)).round()
            Y = torch.matmul(ints, st["w_codes"][:, :K].double().T) * (top / 127) * st["w_scale"].double()
        if not case["r"]:
            return {"Y": Y}
        U = torch.matmul(D * X, st["A"].double().T)
        return {"Y": Y + torch.matmul(U, s * st["B"].double().T), "U": U}
    if k == "nf4_bwd":
        W = _nf4_weight64(st)
    else:
        W = (st["w_codes"][:, :K].double() * st["w_scale"].double()[:, None]).float().bfloat16().double()
    dY = st["dY"].double()
    G = s * torch.matmul(dY, st["B"].double())
    dX = torch.matmul(dY, W) + D * torch.matmul(G, st["A"].double())
    return {"dX": dX, "dA": torch.matmul(G.T, D * X), "dB": s * torch.matmul(dY.T, st["U"].double())}
