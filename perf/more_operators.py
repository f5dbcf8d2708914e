"""Operators between the rank sum and the residual add, as cases to be timed and compared: the branch of a decoder
block (a norm behind the block, its gate, dropout, the residual's scale) with the next block's norm, its backward, and
dropout of the rank sum alone.

With ``own`` false ``run`` computes them in plain torch operations, in 32 bits, rounded once at the end (long sums
in 64); with ``own`` true it calls the framework.  ``exact`` gives the same outputs from the definitions in 64 bits.

The branch: y = rmsnorm(sum_r x_r) * norm_weight (or the sum itself), z = dropout(gate * y), h = residual_scale *
residual + z, norm_out = rmsnorm(h) * weight.  gate_rows: None for no gate, 0 for a gate of its own for every row, G for
a gate [G, N] of which every row serves M / G consecutive rows of the batch.
"""
import math

import numpy as np
import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
LARGEST = 1.2e9    # bytes of the largest listed case; drawn ones stay below
MASK32 = 0xFFFFFFFF


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _case(name, op, W, M, N, dtype, norm=False, gate_rows=None, residual_scale=1.0, p=0.0, keep=False):
    """norm: with a norm behind the block.  keep: the forward stores the rank sum for a backward."""
    return {"name": name, "op": op, "W": W, "M": M, "N": N, "dtype": dtype, "norm": norm, "gate_rows": gate_rows,
            "residual_scale": residual_scale, "p": p, "keep": keep}


def listed():
    return [
        # one token of one request, norms before and after the block: nothing but latency
        _case("norms_token_w2", "branch", 2, 1, 2048, "bf16", norm=True),
        # a decode step of 24 requests over eight ranks
        _case("norms_decode_w8", "branch", 8, 24, 8192, "bf16", norm=True),
        # the framework's own batch size, in training: the rank sum is kept for the backward
        _case("norms_batch_w8", "branch", 8, 512, 8192, "bf16", norm=True, keep=True),
        # a transformer conditioned on each of twelve samples: a gate row per sample, odd number of tokens, short rows
        _case("gate_samples_w1", "branch", 1, 12 * 1111, 1160, "fp16", gate_rows=12, keep=True),
        # dropout before the residual add, long prompts of a training batch, an odd number of tokens
        _case("dropout_norm_w4", "branch", 4, 8191, 8192, "bf16", p=0.1),
        # the gradient of a short sequence, columns not a multiple of 128
        _case("normsgrad_short_w2", "branchgrad", 2, 37, 2056, "bf16", norm=True),
        # the framework's own batch size, backwards
        _case("normsgrad_batch_w8", "branchgrad", 8, 512, 8192, "bf16", norm=True),
        # its fp32 workload, backwards: a learned gate per column, and both paths scaled
        _case("normsgrad_fp32_w4", "branchgrad", 4, 2048, 4096, "fp32", norm=True, gate_rows=1, residual_scale=0.75),
        # the conditioned transformer's gradient: one row of gradients per sample
        _case("gategrad_samples_w1", "branchgrad", 1, 12 * 1111, 1160, "fp16", gate_rows=12),
        # a training micro-batch without tensor parallelism: norms on both sides and dropout, backwards
        _case("dropoutgrad_tokens_w1", "branchgrad", 1, 16389, 4096, "bf16", norm=True, p=0.1),
        # dropout behind a small embedding split over two ranks: nothing but latency
        _case("dropout_embed_w2", "dropout", 2, 61, 1032, "bf16", p=0.1),
        # dropout behind an embedding split over eight ranks
        _case("dropout_embed_w8", "dropout", 8, 4099, 4096, "bf16", p=0.1),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def draw(rng):
    while True:
        op = rng.choice(("branch", "branch", "branchgrad", "branchgrad", "dropout"))
        W = rng.choice((1, 2, 3, 4, 6, 8, 8, 16))
        dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        M, N = int(_log(rng, 1, 8192)), 8 * int(_log(rng, 32, 2048))
        p = rng.choice((0.05, 0.1, 0.2, 0.5))
        if op == "dropout":
            c = _case("", op, W, M, N, dtype, p=p)
        else:
            gate_rows = rng.choice((None, None, 0, 1, 8))
            if gate_rows == 8:  # samples of a batch
                gate_rows = rng.randint(2, 16)
                M = gate_rows * max(1, M // gate_rows)
            c = _case("", op, W, M, N, dtype, rng.random() < 0.7, gate_rows, rng.choice((1.0, 1.0, 0.5, 1.25)),
                      p if rng.random() < 0.4 else 0.0, op == "branch" and rng.random() < 0.4)
        if work(c)["bytes"] < LARGEST:
            del c["name"]
            return c


def _needs_sum(case):
    """The backward reads the stored rank sum for the norm behind the block and for the gate's gradient."""
    return case["norm"] or case["gate_rows"] is not None


def work(case):
    W, M, N, s = case["W"], case["M"], case["N"], SIZE[case["dtype"]]
    full, gate = M * N * s, case["gate_rows"]
    drop = 12 * M * N if case["p"] else 0  # of the generator, by element
    if case["op"] == "dropout":
        return {"bytes": (W + 1) * full, "flops": W * M * N + drop}
    rows = (2 if case["norm"] else 1) * N * s
    gates = 0 if gate is None else (M if gate == 0 else gate) * N
    if case["op"] == "branch":
        return {"bytes": (W + 3 + (1 if case["keep"] else 0)) * full + rows + gates * s, "flops": (W + 10) * M * N + drop}
    grads = (2 if case["norm"] else 1) * N * 4 + gates * (s if gate == 0 else 4)
    return {"bytes": (W + 4 + (1 if _needs_sum(case) else 0)) * full + rows + gates * s + grads,
            "flops": (W + 28) * M * N + drop}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _randn(gen, shape, dtype, sigma):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(sigma)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    t, W, M, N, op = DTYPE[case["dtype"]], case["W"], case["M"], case["N"], case["op"]
    s = {"case": case, "eps": 1e-6}
    # the state of the dropout's generator: a training run's seed and the layer's and step's own offset
    s["seed"] = 0x9E3779B9 * (seed + 1) % 2**62
    s["offset"] = 2**33 * (seed % 1000) + 7
    if op == "dropout":
        s["x"] = _randn(gen, (W, M, N), t, 1.0 / math.sqrt(W))
        s["out"] = torch.empty(M, N, dtype=t, device="cuda")
    else:
        weights = lambda: (torch.rand(N, generator=gen, device="cuda") + 0.5).to(t)  # noqa: E731
        s["weight"], s["norm_weight"] = weights(), weights() if case["norm"] else None
        s["gate"] = None
        if case["gate_rows"] is not None:
            s["gate"] = _randn(gen, (case["gate_rows"] or M, N), t, 0.5)
        # the residual stream has a few columns that are far larger than the others
        loud = torch.where(torch.rand(N, generator=gen, device="cuda") < 0.01, 20.0, 1.0).to(t)
        if op == "branch":
            s["x"] = _randn(gen, (W, M, N), t, 1.0 / math.sqrt(W))
            s["residual"] = _randn(gen, (M, N), t, 1.0).mul_(loud)
            s["residual_out"], s["norm_out"] = torch.empty_like(s["residual"]), torch.empty_like(s["residual"])
            s["sum"] = torch.empty_like(s["residual"]) if case["keep"] else None
        else:
            s["dy"] = _randn(gen, (W, M, N), t, 0.02)
            s["sum"] = _randn(gen, (M, N), t, 1.0) if _needs_sum(case) else None
            s["h"] = _randn(gen, (M, N), t, 1.5).mul_(loud)
            s["dres"] = _randn(gen, (M, N), t, 0.05)
            s["dx"], s["dresidual"] = torch.empty_like(s["h"]), torch.empty_like(s["h"])
            s["dweight"] = torch.empty(N, device="cuda")
            s["dnorm_weight"] = torch.empty(N, device="cuda") if case["norm"] else None
            s["dgate"] = None
            if s["gate"] is not None:
                s["dgate"] = torch.empty_like(s["gate"]) if case["gate_rows"] == 0 else torch.empty_like(s["gate"],
                                                                                                  dtype=torch.float32)
    if own:
        from rank_sum_reduce_gb300 import Branch, Car, Dropout

        s["car"] = Car(W, M, N, case["dtype"])
        s["ranks"] = list((s["dy"] if op == "branchgrad" else s["x"]).unbind(0))
        s["dropout"] = Dropout(case["p"], s["seed"], s["offset"]) if case["p"] else None
        if op != "dropout":
            s["branch"] = Branch(norm_weight=s["norm_weight"], norm_eps=s["eps"], gate=s["gate"],
                                 gate_rows=1 if case["gate_rows"] is None else case["gate_rows"],
                                 residual_scale=case["residual_scale"], dropout=s["dropout"])
        if op == "branchgrad":
            s["workspace"] = torch.empty(s["car"].branch_workspace_bytes(s["branch"]), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _bits(s):
    """Philox4x32-10 (Salmon, Moraes, Dror and Shaw, 2011): 16 bits for every element of [M, N].  Eight consecutive
    elements share one counter; 64-bit products wrap, and their halves are cut out."""
    M, N = s["case"]["M"], s["case"]["N"]
    at = torch.arange(-(-M * N // 8), device="cuda")
    c = [at & MASK32, at >> 32, torch.full_like(at, s["offset"] & MASK32), torch.full_like(at, s["offset"] >> 32)]
    k = [s["seed"] & MASK32, s["seed"] >> 32]
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32 & MASK32) ^ c[1] ^ k[0], b & MASK32, (a >> 32 & MASK32) ^ c[3] ^ k[1], a & MASK32]
        k = [(k[0] + 0x9E3779B9) & MASK32, (k[1] + 0xBB67AE85) & MASK32]
    halves = torch.stack([half for word in c for half in (word & 0xFFFF, word >> 16)], 1)
    return halves.reshape(-1)[:M * N].reshape(M, N)


def _dropped(s, v):
    threshold = round(s["case"]["p"] * 65536)
    if threshold == 0:
        return v
    return torch.where(_bits(s) >= threshold, v * (65536 / (65536 - threshold)), 0.0)


def _gate(s):
    """[M, N] in 32 bits, or None."""
    if s["gate"] is None:
        return None
    return s["gate"].float().repeat_interleave(s["case"]["M"] // s["gate"].shape[0], 0)


def _inverse_rms(v, eps):
    return torch.rsqrt((v * v).mean(-1, keepdim=True) + eps)


def _plain_branch(s):
    c = s["case"]
    t = DTYPE[c["dtype"]]
    acc = s["x"].sum(0, dtype=torch.float32)
    z = acc
    if c["norm"]:
        z = z * _inverse_rms(acc, s["eps"]) * s["norm_weight"].float()
    if s["gate"] is not None:
        z = z * _gate(s)
    h = s["residual"].float() * c["residual_scale"] + _dropped(s, z)
    out = {"residual_out": h.to(t), "norm_out": (h * _inverse_rms(h, s["eps"]) * s["weight"].float()).to(t)}
    if c["keep"]:
        out["sum"] = acc.to(t)
    return out


def _plain_branchgrad(s):
    c = s["case"]
    t, M, N = DTYPE[c["dtype"]], c["M"], c["N"]
    g = s["dy"].sum(0, dtype=torch.float32)
    h, w = s["h"].float(), s["weight"].float()
    r = _inverse_rms(h, s["eps"])
    dh = r * g * w - h * (r * r * r * (g * w * h).mean(-1, keepdim=True)) + s["dres"].float()
    out = {"dweight": (g * h * r).sum(0, dtype=torch.float64).float(), "dresidual": (dh * c["residual_scale"]).to(t)}
    dz = _dropped(s, dh)
    y = u = s["sum"].float() if s["sum"] is not None else None
    if c["norm"]:
        q = _inverse_rms(y, s["eps"])
        u = y * q
        y = u * s["norm_weight"].float()
    if s["gate"] is not None:
        G = s["gate"].shape[0]
        dgate = dz * y
        out["dgate"] = dgate.to(t) if c["gate_rows"] == 0 else dgate.reshape(G, M // G, N).sum(1, dtype=torch.float64).float()
        dz = dz * _gate(s)
    if c["norm"]:
        out["dnorm_weight"] = (dz * u).sum(0, dtype=torch.float64).float()
        v = dz * s["norm_weight"].float()
        dz = q * (v - u * (v * u).mean(-1, keepdim=True))
    out["dx"] = dz.to(t)
    return out


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        if op == "dropout":
            return _dropped(s, s["x"].sum(0, dtype=torch.float32)).to(s["out"].dtype)
        return _plain_branch(s) if op == "branch" else _plain_branchgrad(s)
    if op == "dropout":
        s["car"].reduce_dropout(s["ranks"], s["dropout"], s["out"])
        return s["out"]
    if op == "branch":
        s["car"].reduce_branch_residual_rmsnorm(s["ranks"], s["branch"], s["residual"], s["weight"], s["eps"],
                                                s["residual_out"], s["norm_out"], ar_out=s["sum"])
        out = {"residual_out": s["residual_out"], "norm_out": s["norm_out"]}
        if s["sum"] is not None:
            out["sum"] = s["sum"]
        return out
    s["car"].reduce_branch_residual_rmsnorm_backward(s["ranks"], s["branch"], s["sum"], s["h"], s["weight"], s["eps"],
                                                     s["dres"], s["dx"], s["dresidual"], s["dweight"],
                                                     dnorm_weight=s["dnorm_weight"], dgate=s["dgate"],
                                                     workspace=s["workspace"])
    out = {"dweight": s["dweight"], "dresidual": s["dresidual"]}
    if s["dgate"] is not None:
        out["dgate"] = s["dgate"]
    if s["dnorm_weight"] is not None:
        out["dnorm_weight"] = s["dnorm_weight"]
    out["dx"] = s["dx"]
    return out


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _kept(s):
    """The factor of every element of [M, N], 0 or 1 / (1 - p), from the generator's definition in numpy."""
    c = s["case"]
    drop = round(c["p"] * 65536)
    if drop == 0:
        return 1.0
    n = c["M"] * c["N"]
    index = np.arange((n + 7) // 8, dtype=np.uint64)
    word = np.empty((index.size, 4), dtype=np.uint32)
    word[:, 0], word[:, 1] = index.astype(np.uint32), (index >> np.uint64(32)).astype(np.uint32)
    word[:, 2], word[:, 3] = s["offset"] % 2**32, s["offset"] // 2**32
    key = (s["seed"] % 2**32, s["seed"] // 2**32)
    for r in range(10):
        first = word[:, 0].astype(np.uint64) * np.uint64(0xD2511F53)
        second = word[:, 2].astype(np.uint64) * np.uint64(0xCD9E8D57)
        round_key = [np.uint32((k + r * step) % 2**32) for k, step in zip(key, (0x9E3779B9, 0xBB67AE85))]
        mixed = np.empty_like(word)
        mixed[:, 0] = (second >> np.uint64(32)).astype(np.uint32) ^ word[:, 1] ^ round_key[0]
        mixed[:, 1] = second.astype(np.uint32)
        mixed[:, 2] = (first >> np.uint64(32)).astype(np.uint32) ^ word[:, 3] ^ round_key[1]
        mixed[:, 3] = first.astype(np.uint32)
        word = mixed
    stays = word.astype("<u4").view("<u2").reshape(-1)[:n] >= drop  # the low half of a word first
    factor = torch.from_numpy(stays).reshape(c["M"], c["N"]).cuda().double()
    return factor.mul_(1.0 / (1.0 - drop / 65536))


def _sum64(x):
    acc = torch.zeros(x.shape[1:], dtype=torch.float64, device=x.device)
    for r in range(x.shape[0]):
        acc += x[r]
    return acc


def _rms64(v, eps):
    return torch.sqrt(torch.linalg.vector_norm(v, dim=1, keepdim=True) ** 2 / v.shape[1] + eps)


def exact(case, seed):
    s = prepare(case, seed)
    M, N = case["M"], case["N"]
    kept = _kept(s)
    if case["op"] == "dropout":
        return _sum64(s["x"]) * kept
    gate = None
    if s["gate"] is not None:
        rows = torch.arange(M, device="cuda") * s["gate"].shape[0] // M
        gate = s["gate"].double()[rows]
    w = s["weight"].double()
    w1 = s["norm_weight"].double() if case["norm"] else None
    if case["op"] == "branch":
        acc = _sum64(s["x"])
        z = acc / _rms64(acc, s["eps"]) * w1 if case["norm"] else acc
        if gate is not None:
            z = gate * z
        h = torch.add(kept * z, s["residual"].double(), alpha=case["residual_scale"])
        out = {"residual_out": h, "norm_out": h / _rms64(h, s["eps"]) * w}
        if case["keep"]:
            out["sum"] = acc
        return out
    g, h = _sum64(s["dy"]), s["h"].double()
    rms = _rms64(h, s["eps"])
    u = h / rms
    gw = g * w
    dh = (gw - u * (torch.einsum("mn,mn->m", gw, u) / N)[:, None]) / rms + s["dres"].double()
    out = {"dweight": torch.einsum("mn,mn->n", g, u), "dresidual": case["residual_scale"] * dh}
    dz = kept * dh
    a = s["sum"].double() if s["sum"] is not None else None
    rms1 = _rms64(a, s["eps"]) if case["norm"] else None
    if gate is not None:
        to_gate = dz * (a / rms1 * w1 if case["norm"] else a)
        G = s["gate"].shape[0]
        out["dgate"] = torch.stack([part.sum(0) for part in to_gate.split(M // G)]) if case["gate_rows"] else to_gate
        dz = gate * dz
    if case["norm"]:
        u1 = a / rms1
        out["dnorm_weight"] = torch.einsum("mn,mn->n", dz, u1)
        v = dz * w1
        dz = (v - u1 * (torch.einsum("mn,mn->m", v, u1) / N)[:, None]) / rms1
    out["dx"] = dz
    return out
