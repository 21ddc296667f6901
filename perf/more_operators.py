"""Timed cases of the gated feed-forward block and of the adapters of many
requests, both on frozen 4-bit (NF4) weights.

Kinds of case:

  gated_fwd    H = act(G) o P with G = X deq(Wg)^T + s Ug Bg^T, P = X deq(Wu)^T
               + s Uu Bu^T and [Ug | Uu] = X A^T (A = Ag over Au, B = Bg over
               Bu); with `save` also GU = [G | P] and U = [Ug | Uu], in 16 bits,
               for the backward pass
  gated_bwd    from dH, GU and U: dG = dH o P o act'(G) and dP = dH o act(G),
               rounded to the 16 bits that every gradient of a projection's
               output has here, then dX = dG deq(Wg) + dP deq(Wu) + s (dG Bg)
               Ag + s (dP Bu) Au, dA = s [dG Bg | dP Bu]^T X and dB = s [dG^T Ug
               ; dP^T Uu]
  many_fwd     Y_m = deq(W) x_m + scale_a B_a (A_a x_m) with a = ids[m] the slot
               of token m's adapter in a pool; a token whose id is outside the
               pool gets deq(W) x_m alone
  gated_many   gated_fwd with such a pool of adapters in place of the one

act(x) = x sigma(p(x)): p(x) = x (silu), or 2 sqrt(2 / pi) (x + 0.044715 x^3)
(gelu, whose tanh form this is).

A pool holds the adapters of S slots: A [S, g R, K], B [S, g N, R] (g = 2 for a
gated block, gate before up), a scale and a rank (at most R) per slot.

With `own` false, run() uses elementary torch operations in 32 bits (64 for the
gradients that are rounded in between); with `own` true it calls
bit_quantized_finetuning_nf4_amd.ops.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
ALPHA = 16.0

NF4_BITS = (0xBF800000, 0xBF3239B1, 0xBF066B2E, 0xBECA329E, 0xBE91A24B, 0xBE3D353D, 0xBDBA7869, 0x00000000,
            0x3DA2FB01, 0x3E24CADF, 0x3E7C04DA, 0x3EAD0336, 0x3EE1A4B5, 0x3F1007A9, 0x3F3913B0, 0x3F800000)


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one token through the 7B layer set's gate and up projections with an adapter: latency
        dict(name="gated_token_7b", kind="gated_fwd", M=1, N=11008, K=4096, r=64, act="silu", save=False),
        # a ragged prompt through the 7B block
        dict(name="gated_ragged_7b", kind="gated_fwd", M=333, N=11008, K=4096, r=16, act="silu", save=False),
        # the 65B block in training: the largest call
        dict(name="gated_train_65b", kind="gated_fwd", M=4096, N=22016, K=8192, r=64, act="silu", save=True),
        # the single small linear's sizes, backward
        dict(name="gated_bwd_small", kind="gated_bwd", M=256, N=1024, K=1024, r=8, act="gelu"),
        # the 13B block in training, backward
        dict(name="gated_bwd_13b", kind="gated_bwd", M=2048, N=13824, K=5120, r=64, act="silu"),
        # one token through the 7B query projection with its adapter out of a pool
        dict(name="many_token_7b", kind="many_fwd", M=1, N=4096, K=4096, R=16, slots=8, requests=1, mixed=False,
             bare=False),
        # a decode batch through the 65B query projection, every request with an adapter of its own
        dict(name="many_batch16_65b", kind="many_fwd", M=16, N=8192, K=8192, R=16, slots=16, requests=16, mixed=False,
             bare=False),
        # packed prompts of eleven requests through the 13B down projection, ranks 8 to 64, some without an adapter
        dict(name="many_ragged_13b", kind="many_fwd", M=777, N=5120, K=13824, R=64, slots=7, requests=11, mixed=True,
             bare=True),
        # long prompts of eight requests through the 65B down projection
        dict(name="many_prompts_65b", kind="many_fwd", M=4096, N=8192, K=22016, R=64, slots=8, requests=8, mixed=False,
             bare=False),
        # a decode batch through the 65B block, forty slots
        dict(name="gated_many_32_65b", kind="gated_many", M=32, N=22016, K=8192, R=16, slots=40, requests=32,
             mixed=False, bare=True, act="silu"),
        # prompts of twelve requests through the 13B block
        dict(name="gated_many_prompts_13b", kind="gated_many", M=1200, N=13824, K=5120, R=32, slots=12, requests=12,
             mixed=True, bare=False, act="gelu"),
    ]


def _spread(rng, lo, hi, step):
    """A multiple of `step` between lo and hi, even over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    kind = rng.choice(("gated_fwd", "gated_fwd", "gated_bwd", "many_fwd", "many_fwd", "gated_many"))
    g = 1 if kind == "many_fwd" else 2
    while True:
        M = _spread(rng, 16 if kind == "gated_bwd" else 1, 4096, 1)
        N, K = _spread(rng, 512, 22016, 8), _spread(rng, 512, 22016 if g == 1 else 8192, 64)
        if M * g * N * K <= 4096 * 2 * 22016 * 8192:
            break
    act = rng.choice(("silu", "silu", "gelu"))
    if kind == "gated_fwd":
        return dict(kind=kind, M=M, N=N, K=K, r=rng.choice((0, 8, 16, 32, 64, 128)), act=act, save=rng.random() < 0.5)
    if kind == "gated_bwd":
        return dict(kind=kind, M=M, N=N, K=K, r=rng.choice((8, 16, 32, 64, 128)), act=act)
    R = rng.choice((8, 16, 32, 64, 128))
    case = dict(kind=kind, M=M, N=N, K=K, R=R, slots=_spread(rng, 1, min(64, 1024 // R), 1),
                requests=_spread(rng, 1, min(M, 64), 1), mixed=rng.random() < 0.5, bare=rng.random() < 0.3)
    return dict(case, act=act) if kind == "gated_many" else case


def _slots_of(case):
    """The slot of each request, -1 for one without an adapter."""
    return [-1 if case["bare"] and i % 5 == 4 else i % case["slots"] for i in range(case["requests"])]


def _rank_of(case, slot):
    return max(8, case["R"] >> (slot % 3) if case["mixed"] else case["R"])


def work(case):
    k, M, N, K = case["kind"], case["M"], case["N"], case["K"]
    g = 1 if k == "many_fwd" else 2
    weight = g * N * K / 2 + g * N * K / 64 + g * N * K / 4096
    flops = 2 * M * g * N * K
    if k == "gated_bwd":
        r = case["r"]
        return {"bytes": int(weight + 2 * M * K + 6 * M * N + 4 * M * r + 4 * r * (N + K) + 2 * M * K + 8 * r * (N + K)),
                "flops": flops + 8 * M * r * (N + K)}
    if k == "gated_fwd":
        r = case["r"]
        out = 2 * M * N + (4 * M * N + 4 * M * r if case["save"] else 0)
        return {"bytes": int(weight + 2 * M * K + 4 * r * (N + K) + out), "flops": flops + 4 * M * r * (N + K)}
    slots = _slots_of(case)
    ranks = sum(_rank_of(case, s) for s in set(slots) if s >= 0)
    r = sum(_rank_of(case, s) for s in slots if s >= 0) / len(slots)
    return {"bytes": int(weight + 2 * M * K + 2 * g * ranks * (N + K) + 2 * M * N + 4 * M),
            "flops": int(flops + 2 * M * r * g * (N + K))}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _normal(gen, shape, std):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).mul_(std).to(torch.bfloat16)


def _nf4(gen, N, K):
    # uniform codes (the levels are normal quantiles), block constants spread below their group's largest
    blocks = N * K // 64
    return (torch.randint(0, 256, (N * K // 2,), generator=gen, device=DEV, dtype=torch.uint8),
            (torch.randn(blocks, generator=gen, device=DEV) * 25 + 160).clamp_(80, 255).to(torch.uint8),
            torch.rand((blocks + 255) // 256, generator=gen, device=DEV) * 0.02 + 0.07)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    k, M, N, K = case["kind"], case["M"], case["N"], case["K"]
    g = 1 if k == "many_fwd" else 2
    # hidden states of a size that gives the projections' outputs one of about 1
    st = {"case": case, "W": [_nf4(gen, N, K) for _ in range(g)], "X": _normal(gen, (M, K), 25.0 / math.sqrt(K))}
    if k in ("gated_fwd", "gated_bwd"):
        r = case["r"]
        st["A"] = _normal(gen, (2 * r, K), 0.02) if r else None
        st["B"] = _normal(gen, (2 * N, r), 0.02) if r else None
        if k == "gated_bwd":
            st["dH"] = _normal(gen, (M, N), 1.0)
            st["GU"] = _normal(gen, (M, 2 * N), 1.5)
            st["U"] = _normal(gen, (M, 2 * r), 0.5)
        return st
    S, R = case["slots"], case["R"]
    st["A"], st["B"] = _normal(gen, (S, g * R, K), 0.02), _normal(gen, (S, g * N, R), 0.02)
    ranks = [_rank_of(case, s) for s in range(S)]
    st["rank"] = torch.tensor(ranks, dtype=torch.int32, device=DEV)
    # a slot of a smaller rank holds zeros past it
    live = torch.arange(R, device=DEV)[None, :] < st["rank"][:, None]
    st["A"] *= live.repeat(1, g)[:, :, None]
    st["B"] *= live[:, None, :]
    st["scale"] = ALPHA / st["rank"].float()
    # requests of different lengths, one after the other
    cuts = torch.randperm(M - 1, generator=gen, device=DEV)[:case["requests"] - 1].sort().values + 1
    request = (torch.arange(M, device=DEV)[:, None] >= cuts[None, :]).sum(1)
    st["ids"] = torch.tensor(_slots_of(case), dtype=torch.int32, device=DEV)[request]
    return st


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------

def _weight(q, N, K):
    codes, absmax_q, group_scale = q
    levels = torch.from_numpy(np.array(NF4_BITS, dtype=np.uint32).view(np.float32)).to(DEV)
    nibbles = torch.stack((codes & 15, codes >> 4), -1).reshape(-1, 64).long()
    q8 = (torch.arange(256, device=DEV, dtype=torch.float64) / 255).float()
    t = q8[absmax_q.long()] * group_scale[torch.arange(absmax_q.numel(), device=DEV) // 256]
    return (levels[nibbles] * t[:, None]).to(torch.bfloat16).float().view(N, K)


C3 = 0.044715


def _gate(x, act):
    """sigma(p(x)) and p'(x)."""
    if act == "silu":
        return 1 / (1 + torch.exp(-x)), torch.ones_like(x)
    c = 2 * math.sqrt(2 / math.pi)
    return 1 / (1 + torch.exp(-c * (x + C3 * x * x * x))), c * (1 + 3 * C3 * x * x)


def _pool_term(st, g):
    """[M, g, N] of scale B_a (A_a x): every slot's ranks side by side, the other slots' masked."""
    c = st["case"]
    S, R, N = c["slots"], c["R"], c["N"]
    u = (st["X"].float() @ st["A"].float().view(S * g * R, -1).t()).view(-1, S, g, R)
    mine = st["ids"][:, None] == torch.arange(S, device=DEV)[None, :]
    u = u * (mine * st["scale"][None, :])[:, :, None, None]
    b = st["B"].float().view(S, g, N, R)
    if g == 1:
        return (u.reshape(-1, S * R) @ b.permute(0, 3, 1, 2).reshape(S * R, N))[:, None]
    return torch.stack((u[:, :, 0].reshape(-1, S * R) @ b[:, 0].transpose(1, 2).reshape(S * R, N),
                        u[:, :, 1].reshape(-1, S * R) @ b[:, 1].transpose(1, 2).reshape(S * R, N)), 1)


def _plain(st):
    c = st["case"]
    k, N, K = c["kind"], c["N"], c["K"]
    X = st["X"].float()
    if k == "many_fwd":
        return {"Y": (X @ _weight(st["W"][0], N, K).t() + _pool_term(st, 1)[:, 0]).to(torch.bfloat16)}
    if k == "gated_bwd":
        r = c["r"]
        s = ALPHA / r
        G, P, dH = st["GU"][:, :N].double(), st["GU"][:, N:].double(), st["dH"].double()
        sg, dp = _gate(G, c["act"])
        dG = (dH * P * (sg + G * sg * (1 - sg) * dp)).to(torch.bfloat16).float()
        dP = (dH * G * sg).to(torch.bfloat16).float()
        A, B, U = st["A"].float(), st["B"].float(), st["U"].float()
        Tg, Tp = s * (dG @ B[:N]), s * (dP @ B[N:])
        dX = dG @ _weight(st["W"][0], N, K) + dP @ _weight(st["W"][1], N, K) + Tg @ A[:r] + Tp @ A[r:]
        return {"dX": dX.to(torch.bfloat16), "dA": torch.cat((Tg.t() @ X, Tp.t() @ X)),
                "dB": s * torch.cat((dG.t() @ U[:, :r], dP.t() @ U[:, r:]))}
    G, P = X @ _weight(st["W"][0], N, K).t(), X @ _weight(st["W"][1], N, K).t()
    U = None
    if k == "gated_many":
        term = _pool_term(st, 2)
        G, P = G + term[:, 0], P + term[:, 1]
    elif c["r"]:
        r = c["r"]
        U = X @ st["A"].float().t()
        G = G + ALPHA / r * (U[:, :r] @ st["B"][:N].float().t())
        P = P + ALPHA / r * (U[:, r:] @ st["B"][N:].float().t())
    out = {"H": (G * _gate(G, c["act"])[0] * P).to(torch.bfloat16)}
    if k == "gated_fwd" and c["save"]:
        out["GU"] = torch.cat((G, P), 1).to(torch.bfloat16)
        if U is not None:
            out["U"] = U.to(torch.bfloat16)
    return out


# --------------------------------------------------------------------------
# the framework's operators
# --------------------------------------------------------------------------

def _framework(st):
    from bit_quantized_finetuning_nf4_amd import ops

    c = st["case"]
    k = c["kind"]
    qs = [ops.QuantizedWeight(c["N"], c["K"], *w) for w in st["W"]]
    if k == "gated_bwd":
        dX, dA, dB = ops.gated_bwd(qs, st["X"], st["dH"], st["GU"], st["A"], st["B"], ALPHA, act=c["act"], U=st["U"])
        return {"dX": dX, "dA": dA, "dB": dB}
    if k == "gated_fwd":
        if not c["save"]:
            return {"H": ops.gated_fwd(qs, st["X"], st["A"], st["B"], ALPHA, act=c["act"])}
        H, GU, U = ops.gated_fwd(qs, st["X"], st["A"], st["B"], ALPHA, act=c["act"], save=True)
        return {"H": H, "GU": GU, "U": U} if c["r"] else {"H": H, "GU": GU}
    pool = ops.AdapterPool(st["A"], st["B"], st["scale"], st["rank"])
    if k == "gated_many":
        return {"H": ops.gated_many_fwd(qs, st["X"], pool, st["ids"], act=c["act"])}
    return {"Y": ops.many_fwd(qs[0], st["X"], pool, st["ids"])}


def run(state):
    if own:
        return _framework(state)
    return _plain(state)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _weight64(q, N, K):
    codes, absmax_q, group_scale = q
    out = torch.empty(N * K, device=DEV, dtype=torch.float64)
    levels = torch.from_numpy(np.array(NF4_BITS, dtype=np.uint32).view(np.float32).astype(np.float64)).to(DEV)
    # a stored value is the fp32 product of fp32 numbers, rounded to bf16: products of two 24-bit numbers are exact in 64 bits
    scale = (absmax_q.double() / 255).float().double() * group_scale.double().repeat_interleave(256)[:absmax_q.numel()]
    scale = scale.float().double().repeat_interleave(32)
    out[0::2] = (levels[(codes % 16).int()] * scale).float().bfloat16().double()
    out[1::2] = (levels[(codes // 16).int()] * scale).float().bfloat16().double()
    return out.view(N, K)


def _act64(x, act):
    """act and its derivative: the tanh form of gelu, the logistic form of silu."""
    if act == "silu":
        s = torch.sigmoid(x)
        return x * s, s * (1 + x * (1 - s))
    z = math.sqrt(2 / math.pi) * (x + C3 * x ** 3)
    t = torch.tanh(z)
    return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * C3 * x * x)


def exact(case, seed):
    st = prepare(case, seed)
    k, N, K, M = case["kind"], case["N"], case["K"], case["M"]
    X = st["X"].double()
    if k == "gated_bwd":
        r = case["r"]
        s = ALPHA / r
        a, da = _act64(st["GU"][:, :N].double(), case["act"])
        dY = [(st["dH"].double() * st["GU"][:, N:].double() * da).bfloat16().double(),
              (st["dH"].double() * a).bfloat16().double()]
        dX = torch.zeros((M, K), device=DEV, dtype=torch.float64)
        dA, dB = [], []
        for i in range(2):
            A, B = st["A"][i * r:(i + 1) * r].double(), st["B"][i * N:(i + 1) * N].double()
            T = s * torch.matmul(dY[i], B)
            dX += torch.matmul(dY[i], _weight64(st["W"][i], N, K)) + torch.matmul(T, A)
            dA.append(torch.matmul(T.T, X))
            dB.append(s * torch.matmul(dY[i].T, st["U"][:, i * r:(i + 1) * r].double()))
        return {"dX": dX, "dA": torch.cat(dA), "dB": torch.cat(dB)}
    out, U = [], []
    for i in range(len(st["W"])):
        Y = torch.matmul(X, _weight64(st["W"][i], N, K).T)
        if k == "gated_fwd" and case["r"]:
            r = case["r"]
            U.append(torch.matmul(X, st["A"][i * r:(i + 1) * r].double().T))
            Y += ALPHA / r * torch.matmul(U[-1], st["B"][i * N:(i + 1) * N].double().T)
        elif k != "gated_fwd":
            R = case["R"]
            for slot in range(case["slots"]):
                at = torch.nonzero(st["ids"] == slot).flatten()
                A, B = st["A"][slot, i * R:(i + 1) * R].double(), st["B"][slot, i * N:(i + 1) * N].double()
                Y[at] += st["scale"][slot].double() * torch.matmul(torch.matmul(X[at], A.T), B.T)
        out.append(Y)
    if k == "many_fwd":
        return {"Y": out[0]}
    res = {"H": _act64(out[0], case["act"])[0] * out[1]}
    if k == "gated_fwd" and case["save"]:
        res["GU"] = torch.cat(out, 1)
        if U:
            res["U"] = torch.cat(U, 1)
    return res
