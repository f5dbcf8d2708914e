"""The operators next to the rank sum, as cases to be timed and compared: the fused reduce + residual + RMSNorm
with an 8-bit output, its backward, and the rank sum of many gradient tensors with their global norm and clipping.

With ``own`` false ``run`` computes them in plain torch operations, in 32 bits, rounded once at the end (long sums
in 64); with ``own`` true it calls the framework.  ``exact`` gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
GROUP = {"row": None, "group128": 128, "mx32": 32, "static": None}
E4M3_MAX = 448.0
FLOOR = 2.0**-126  # the smallest scale
LARGEST = 3.6e9    # bytes of the largest listed case; drawn ones stay below


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _norm8(name, W, M, N, dtype, kind):
    return {"name": name, "op": "norm8", "W": W, "M": M, "N": N, "dtype": dtype, "kind": kind}


def _normgrad(name, W, M, N, dtype, skip):
    return {"name": name, "op": "normgrad", "W": W, "M": M, "N": N, "dtype": dtype, "skip": skip}


def _grads(name, W, layers, hidden, inner, vocab, dtype, mixed, odd, clip):
    return {"name": name, "op": "grads", "W": W, "layers": layers, "hidden": hidden, "inner": inner, "vocab": vocab,
            "dtype": dtype, "mixed": mixed, "odd": odd, "clip": clip}


def listed():
    return [
        # one token of one request, two ranks: nothing but latency
        _norm8("norm8_token_w2", 2, 1, 2048, "bf16", "row"),
        # a decode step of 24 requests over eight ranks, block-scaled for the tensor cores
        _norm8("norm8_decode_w8", 8, 24, 8192, "bf16", "mx32"),
        # a prefill chunk: the framework's own batch size
        _norm8("norm8_prefill_w8", 8, 512, 8192, "bf16", "group128"),
        # long prompts, an odd number of tokens
        _norm8("norm8_prompts_w4", 4, 8191, 8192, "bf16", "row"),
        # the gradient of a short sequence, columns not a multiple of 128
        _normgrad("normgrad_short_w2", 2, 37, 2056, "bf16", True),
        # the framework's own batch size, backwards
        _normgrad("normgrad_batch_w8", 8, 512, 8192, "bf16", True),
        # its fp32 workload, backwards; the last norm of a model has no skip path
        _normgrad("normgrad_fp32_w4", 4, 2048, 4096, "fp32", False),
        # a training micro-batch without tensor parallelism, odd number of tokens
        _normgrad("normgrad_tokens_w1", 1, 16389, 4096, "bf16", True),
        # an adapter's few gradients: nothing but latency
        _grads("grads_adapter_w2", 2, 2, 64, 96, 0, "bf16", False, False, True),
        # one block's gradients, norm weights in fp32, over the limit
        _grads("grads_block_w4", 4, 1, 2048, 8192, 0, "bf16", True, False, True),
        # fp32 gradients without data parallelism, every tensor of odd size, over the limit
        _grads("grads_odd_w1", 1, 12, 513, 1365, 1000, "fp32", False, True, True),
        # a whole model's gradients over eight ranks, under the limit
        _grads("grads_model_w8", 8, 2, 2048, 8192, 32000, "bf16", True, False, False),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def draw(rng):
    while True:
        op = rng.choice(("norm8", "normgrad", "grads"))
        W = rng.choice((1, 2, 3, 4, 6, 8, 8, 16))
        dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        if op == "grads":
            c = _grads("", W, rng.randint(1, 6), int(_log(rng, 32, 2048)), int(_log(rng, 64, 8192)),
                       rng.choice((0, int(_log(rng, 100, 32000)))), dtype, rng.random() < 0.5, rng.random() < 0.5,
                       rng.random() < 0.7)
        else:
            M, N = int(_log(rng, 1, 8192)), 8 * int(_log(rng, 32, 2048))
            if op == "norm8":
                c = _norm8("", W, M, N, dtype, rng.choice(("row", "group128", "mx32", "static")))
            else:
                c = _normgrad("", W, M, N, dtype, rng.random() < 0.8)
        if work(c)["bytes"] < LARGEST:
            del c["name"]
            return c


def _tensor_sizes(case):
    """Elements of the gradient tensors of a decoder of that shape: [(elements, is a norm weight)]."""
    h, f, more = case["hidden"], case["inner"], 1 if case["odd"] else 0
    sizes = []
    for _ in range(case["layers"]):
        sizes += [(h, True), (3 * h * h, False), (h * h, False), (h, True), (2 * f * h, False), (f * h, False)]
    sizes.append((h, True))
    if case["vocab"]:
        sizes.append((case["vocab"] * h, False))
    return [(n + more, is_norm) for n, is_norm in sizes]


def _buckets(case):
    """{type: elements of its tensors}: the norm weights' gradients are fp32 where the case is mixed."""
    got = {}
    for n, is_norm in _tensor_sizes(case):
        got.setdefault("fp32" if is_norm and case["mixed"] else case["dtype"], []).append(n)
    return got


def work(case):
    W = case["W"]
    if case["op"] == "grads":
        totals = {t: sum(v) for t, v in _buckets(case).items()}
        return {"bytes": sum(n * SIZE[t] * (W + 1) for t, n in totals.items()) + 4,
                "flops": sum(totals.values()) * (W + 3)}
    M, N, s = case["M"], case["N"], SIZE[case["dtype"]]
    if case["op"] == "norm8":
        width = GROUP[case["kind"]] or N
        scales = 4 if case["kind"] == "static" else M * -(-N // width) * (1 if case["kind"] == "mx32" else 4)
        return {"bytes": (W + 2) * M * N * s + N * s + M * N + scales, "flops": (W + 7) * M * N}
    return {"bytes": (W + 2 + (1 if case["skip"] else 0)) * M * N * s + N * s + 4 * N, "flops": (W + 12) * M * N}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _randn(gen, shape, dtype, sigma):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(sigma)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    t, W, op = DTYPE[case["dtype"]], case["W"], case["op"]
    s = {"case": case}
    if op == "grads":
        # flat buckets of one type, one per rank (rows padded so that each starts on its own line), tensors in a row
        scale = 1024.0 if case["dtype"] == "fp16" else 1.0  # gradients in 16 bits are scaled against underflow
        s.update(scale=1.0 / (W * scale), max_norm=1.0, buckets=[])
        n_all = sum(n for n, _ in _tensor_sizes(case))
        sigma = scale * (4.0 if case["clip"] else 0.5) * math.sqrt(W / n_all)
        for name, sizes in _buckets(case).items():
            total = sum(sizes)
            flat = _randn(gen, (W, -(-total // 128) * 128), DTYPE[name], sigma)
            s["buckets"].append({"sizes": sizes, "x": flat[:, :total], "out": torch.empty_like(flat[0])[:total]})
        s["norm"] = torch.empty(1, device="cuda")
        if own:
            from rank_sum_reduce_gb300 import Grads

            split = lambda v, b: list(v.split(b["sizes"]))  # noqa: E731
            s["grads"] = Grads([sum((split(b["x"][r], b) for b in s["buckets"]), []) for r in range(W)],
                               sum((split(b["out"], b) for b in s["buckets"]), []))
        return s
    M, N = case["M"], case["N"]
    s["weight"] = (torch.rand(N, generator=gen, device="cuda") + 0.5).to(t)
    s["eps"] = 1e-6
    # the residual stream has a few columns that are far larger than the others
    loud = torch.where(torch.rand(N, generator=gen, device="cuda") < 0.01, 20.0, 1.0).to(t)
    if op == "norm8":
        s["x"] = _randn(gen, (W, M, N), t, 1.0 / math.sqrt(W))
        s["residual"] = _randn(gen, (M, N), t, 1.0).mul_(loud)
        s["residual_out"] = torch.empty_like(s["residual"])
        s["q"] = torch.empty(M, N, dtype=torch.float8_e4m3fn, device="cuda")
        if case["kind"] == "static":
            s["scales"] = torch.full((1,), 0.1, device="cuda")  # found by calibration; the loudest values saturate
        else:
            shape = (M, -(-N // (GROUP[case["kind"]] or N)))
            s["scales"] = torch.empty(shape, device="cuda", dtype=torch.uint8 if case["kind"] == "mx32" else torch.float32)
    else:
        s["dy"] = _randn(gen, (W, M, N), t, 0.02)
        s["h"] = _randn(gen, (M, N), t, 1.5).mul_(loud)
        s["dres"] = _randn(gen, (M, N), t, 0.05) if case["skip"] else None
        s["dx"] = torch.empty_like(s["h"])
        s["dweight"] = torch.empty(N, device="cuda")
    if own:
        from rank_sum_reduce_gb300 import Car

        s["car"] = Car(W, M, N, case["dtype"])
        if op == "norm8":
            s["ranks"] = list(s["x"].unbind(0))
        else:
            s["ranks"] = list(s["dy"].unbind(0))
            s["workspace"] = torch.empty(s["car"].backward_workspace_bytes, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _values(scales):
    """e8m0 exponents as the powers of two that they stand for."""
    return scales.view(torch.float8_e8m0fnu) if scales.dtype == torch.uint8 else scales


def _groups(y, width):
    """[M, N] as [M, groups, width], the last group filled up with zeros."""
    M, N = y.shape
    return torch.nn.functional.pad(y, (0, -N % width)).reshape(M, -1, width)


def _plain_norm8(s):
    c = s["case"]
    t = DTYPE[c["dtype"]]
    h = s["x"].sum(0, dtype=torch.float32) + s["residual"].float()
    y = h * s["weight"].float() * torch.rsqrt((h * h).mean(-1, keepdim=True) + s["eps"])
    if c["kind"] == "static":
        q = (y / s["scales"]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        return {"residual_out": h.to(t), "q": q}
    yg = _groups(y, GROUP[c["kind"]] or c["N"])
    scale = (yg.abs().amax(-1) / E4M3_MAX).clamp_min(FLOOR)
    stored = scale
    if c["kind"] == "mx32":  # the next power of two, as its biased exponent
        bits = scale.view(torch.int32)
        stored = ((bits >> 23) + ((bits & 0x7FFFFF) != 0)).to(torch.uint8)
        scale = (stored.to(torch.int32) << 23).view(torch.float32)
    q = (yg / scale[..., None]).reshape(c["M"], -1)[:, : c["N"]].to(torch.float8_e4m3fn)
    return {"residual_out": h.to(t), "q": q, "scales": _values(stored)}


def _plain_normgrad(s):
    c = s["case"]
    g = s["dy"].sum(0, dtype=torch.float32)
    h, w = s["h"].float(), s["weight"].float()
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + s["eps"])
    gw = g * w
    dx = r * gw - h * (r * r * r * (gw * h).mean(-1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(DTYPE[c["dtype"]]), "dweight": (g * h * r).sum(0, dtype=torch.float64).float()}


def _plain_grads(s):
    sums = [b["x"].sum(0, dtype=torch.float32) * s["scale"] for b in s["buckets"]]
    norm = torch.stack([(v * v).sum(dtype=torch.float64) for v in sums]).sum().sqrt()
    coef = (s["max_norm"] / (norm + 1e-6)).clamp_max(1.0).float()
    return {"norm": norm.float().reshape(1), "grads": [(v * coef).to(b["x"].dtype) for v, b in zip(sums, s["buckets"])]}


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return _plain_norm8(s) if op == "norm8" else _plain_normgrad(s) if op == "normgrad" else _plain_grads(s)
    if op == "grads":
        s["grads"].reduce_clip(s["scale"], s["max_norm"], s["norm"], once=True)
        return {"norm": s["norm"], "grads": [b["out"] for b in s["buckets"]]}
    if op == "normgrad":
        s["car"].reduce_residual_rmsnorm_backward(s["ranks"], s["h"], s["weight"], s["eps"], s["dres"], s["dx"],
                                                  s["dweight"], workspace=s["workspace"])
        return {"dx": s["dx"], "dweight": s["dweight"]}
    s["car"].reduce_residual_rmsnorm_quant(s["ranks"], s["residual"], s["weight"], s["eps"], s["case"]["kind"],
                                           s["residual_out"], s["q"], s["scales"])
    out = {"residual_out": s["residual_out"], "q": s["q"]}
    if s["case"]["kind"] != "static":
        out["scales"] = _values(s["scales"])
    return out


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _sum64(x):
    acc = torch.zeros(x.shape[1:], dtype=torch.float64, device=x.device)
    for r in range(x.shape[0]):
        acc += x[r]
    return acc


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "grads":
        sums = [_sum64(b["x"]) / (1.0 / s["scale"]) for b in s["buckets"]]
        norm = math.sqrt(sum(float(torch.dot(v, v)) for v in sums))
        factor = min(1.0, s["max_norm"] / (norm + 1e-6))
        return {"norm": torch.tensor([norm], dtype=torch.float64), "grads": [v.mul_(factor) for v in sums]}
    w = s["weight"].double()
    N = case["N"]
    if case["op"] == "normgrad":
        g, h = _sum64(s["dy"]), s["h"].double()
        r = 1.0 / torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / N + s["eps"])
        u = h * r  # the normalised row; y = u * w
        gw = g * w
        dx = r * (gw - u * ((gw * u).sum(1, keepdim=True) / N))
        if s["dres"] is not None:
            dx += s["dres"].double()
        return {"dx": dx, "dweight": torch.einsum("mn,mn->n", g, u)}
    h = _sum64(s["x"]) + s["residual"].double()
    y = h / torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / N + s["eps"]) * w
    if case["kind"] == "static":
        return {"residual_out": h, "q": torch.clamp(y / s["scales"].double(), -E4M3_MAX, E4M3_MAX)}
    width = GROUP[case["kind"]] or N
    q, scales = torch.empty_like(y), []
    for at in range(0, N, width):
        part = y[:, at:at + width]
        scale = torch.clamp(part.abs().max(dim=1).values / E4M3_MAX, min=FLOOR)
        if case["kind"] == "mx32":
            scale = torch.exp2(torch.ceil(torch.log2(scale)))
        q[:, at:at + width] = part / scale[:, None]
        scales.append(scale)
    # q: the quotient before its rounding to e4m3.  A power of two next to a border has no value of its own.
    return {"residual_out": h, "q": q, "scales": None if case["kind"] == "mx32" else torch.stack(scales, 1)}
