"""Shared by the tests of a block's branch and of dropout: the generator in numpy, and the formulas in 64 bits with bounds.

Tolerances (DELTA and half: see operator_checks).  DELTA bounds what fp32 arithmetic can lose of a value normalised over a
row; the gate, the dropout's scale and one more weight add 3 products to the 25.5 roundings counted there: still under 32.

Forward: y loses DELTA of itself, so h = s res + z loses b = DELTA |z| + 2^-23 |h| (one fused product and sum).  The norm of
h then loses DELTA of itself, |r w| b, and through r, whose relative change is at most r times the root mean square of b.

Backward: dh as the fused op's backward (test_norm_backward_gpu).  What is computed from a value x with a bound b by
products carries b through them, with 2^-23 of the result for up to two products.  Sums over rows: at most 64 rows in a
register or a team, 16 teams, 16 partials in a thread and 32 of a block: 128 roundings of 2^-24, 2^-17 of the sum of the
absolute terms (half a step of which is the fp32 output's own)."""
import numpy as np
import torch

from operator_checks import DELTA, DEV, TINY, TORCH_DTYPE, assert_within, half, randn, rank_sum

M0, M1, W0, W1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85


def philox(counter, key):
    """Philox4x32-10: counter [n, 4] and key [2] of 32-bit words -> [n, 4]."""
    c = np.asarray(counter, dtype=np.uint64)
    k0, k1 = (int(k) for k in key)
    for _ in range(10):
        a, b = c[:, 0] * np.uint64(M0), c[:, 2] * np.uint64(M1)
        low, shift = np.uint64(0xFFFFFFFF), np.uint64(32)
        c = np.stack([(b >> shift) ^ c[:, 1] ^ np.uint64(k0), b & low, (a >> shift) ^ c[:, 3] ^ np.uint64(k1), a & low], 1)
        k0, k1 = (k0 + W0) % 2**32, (k1 + W1) % 2**32
    return c.astype(np.uint32)


def threshold(p):
    return int(np.floor(float(np.float32(p)) * 65536 + 0.5))


def factor(M, N, p, seed, offset, device=DEV):
    """[M, N] in 64 bits: 0 where an element is dropped, 65536 / (65536 - t) elsewhere."""
    t = threshold(p)
    n = M * N
    at = np.arange(-(-n // 8), dtype=np.uint64)
    words = np.stack([at % 2**32, at >> np.uint64(32), np.full_like(at, offset % 2**32), np.full_like(at, offset // 2**32)], 1)
    w = philox(words, (seed % 2**32, seed // 2**32))
    bits = np.stack([w & 0xFFFF, w >> 16], 2).reshape(-1)[:n]
    kept = torch.from_numpy((bits >= t).astype(np.float64)).reshape(M, N).to(device)
    return kept * (65536.0 / (65536 - t) if t < 65536 else 0.0)


class Case:
    """A branch with inputs.  gate_rows: None, 0 (a row for every row) or G."""

    def __init__(self, W, M, N, dtype, norm=True, gate_rows=None, scale=1.0, p=0.0, seed=0, skip=True, eps=1e-6):
        g = torch.Generator(DEV).manual_seed(1000 * W + M + N + seed)
        self.W, self.M, self.N, self.dtype, self.eps, self.norm_eps = W, M, N, dtype, eps, 3 * eps
        t = TORCH_DTYPE[dtype]
        weight = lambda: (torch.rand(N, generator=g, device=DEV) + 0.5).to(t)  # noqa: E731
        self.xs = [randn(g, (M, N), dtype, W**-0.5) for _ in range(W)]
        self.residual, self.weight = randn(g, (M, N), dtype, 1.3), weight()
        self.norm_weight = weight() if norm else None
        self.gate = None if gate_rows is None else randn(g, (gate_rows or M, N), dtype, 0.7)
        self.gate_rows, self.scale, self.p = gate_rows, scale, p
        self.seed, self.offset = 2**63 + 12345 * (seed + 1), 2**40 + 17 * M + seed
        self.dys = [randn(g, (M, N), dtype, 0.1) for _ in range(W)]
        self.a, self.h = randn(g, (M, N), dtype), randn(g, (M, N), dtype, 1.5)
        self.dres = randn(g, (M, N), dtype, 0.2) if skip else None
        self._factor = None

    def factor(self):
        if self._factor is None:
            self._factor = 1.0 if threshold(self.p) == 0 else factor(self.M, self.N, self.p, self.seed, self.offset)
        return self._factor

    def branch(self, car, **changes):
        drop = car.Dropout(self.p, self.seed, self.offset) if self.p else None
        return car.Branch(**{**dict(norm_weight=self.norm_weight, norm_eps=self.norm_eps, gate=self.gate,
                                    gate_rows=1 if self.gate_rows is None else self.gate_rows, residual_scale=self.scale,
                                    dropout=drop), **changes})

    def gates(self):
        if self.gate is None:
            return 1.0
        return self.gate.double().repeat_interleave(self.M // self.gate.shape[0], 0)

    # -- forward ------------------------------------------------------------
    def forward(self):
        """{name: (value, bound without the output's rounding)} in 64 bits."""
        acc = rank_sum(self.xs).double()
        y = acc
        if self.norm_weight is not None:
            y = acc / torch.sqrt((acc * acc).mean(1, keepdim=True) + self.norm_eps) * self.norm_weight.double()
        z = y * self.gates() * self.factor()
        h = self.scale * self.residual.double() + z
        b = DELTA * z.abs() + 2.0**-23 * h.abs()
        r = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + self.eps)
        w = self.weight.double()
        out = h * r * w
        bn = DELTA * out.abs() + (r * w).abs() * b + out.abs() * r * (b * b).mean(1, keepdim=True).sqrt()
        return {"ar": (acc, torch.zeros_like(acc)), "residual_out": (h, b), "norm_out": (out, bn)}

    def check_forward(self, got):
        want = self.forward()
        for name, t in got.items():
            if t is not None:
                v, b = want[name]
                assert_within(t, v, half(self.dtype) * v.abs() + (1 + half(self.dtype)) * b + TINY[self.dtype], name)

    # -- backward -----------------------------------------------------------
    def backward(self):
        g, h, w = rank_sum(self.dys).double(), self.h.double(), self.weight.double()
        r = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + self.eps)
        u = h * r
        gwu = g * w * u
        m = gwu.mean(1, keepdim=True)
        d = torch.zeros_like(h) if self.dres is None else self.dres.double()
        dh = r * (g * w - u * m) + d
        b = DELTA * ((r * g * w).abs() + d.abs() + 2 * (r * u).abs() * gwu.abs().mean(1, keepdim=True) + (r * u * m).abs())
        out = {"dweight": ((g * u).sum(0), 2.0**-17 * (g * u).abs().sum(0)),
               "dresidual": (self.scale * dh, abs(self.scale) * b + 2.0**-23 * (self.scale * dh).abs())}
        f, gate = self.factor(), self.gates()
        dz, bz = f * dh, f * (b + 2.0**-23 * dh.abs())
        u1 = self.a.double()
        w1, q = 1.0, 1.0
        if self.norm_weight is not None:
            q = 1 / torch.sqrt((u1 * u1).mean(1, keepdim=True) + self.norm_eps)
            u1, w1 = u1 * q, self.norm_weight.double()
        t = dz * u1
        bt = bz * u1.abs() + DELTA * t.abs()
        if self.gate is not None:
            v, bv = t * w1, bt * w1 + 2.0**-23 * (t * w1).abs()
            if self.gate_rows:
                rows = lambda x: x.reshape(self.gate_rows, -1, self.N).sum(1)  # noqa: E731
                out["dgate"] = (rows(v), rows(bv) + 2.0**-17 * rows(v.abs()))
            else:
                out["dgate"] = (v, bv)
        v = dz * gate * w1
        bv = bz * (abs(gate) if self.gate is None else gate.abs()) * w1 + 2.0**-22 * v.abs()
        if self.norm_weight is not None:
            gt = gate * t
            out["dnorm_weight"] = (gt.sum(0), ((gate if self.gate is None else gate.abs()) * bt).sum(0) + 2.0**-17 * gt.abs().sum(0))
            vu = v * u1
            mean = vu.mean(1, keepdim=True)
            dx = q * (v - u1 * mean)
            bx = DELTA * ((q * v).abs() + 2 * (q * u1).abs() * vu.abs().mean(1, keepdim=True) + (q * u1 * mean).abs())
            bx = bx + q * bv + (q * u1).abs() * (bv * u1.abs()).mean(1, keepdim=True)
            out["dx"] = (dx, bx)
        else:
            out["dx"] = (v, bv)
        return out

    def check_backward(self, got):
        want = self.backward()
        for name, t in got.items():
            if t is not None:
                v, b = want[name]
                if t.dtype == torch.float32 and self.dtype != "fp32":
                    assert_within(t, v, b, name)
                else:
                    assert_within(t, v, half(self.dtype) * v.abs() + (1 + half(self.dtype)) * b + TINY[self.dtype], name)

    def grads(self, empty):
        """Outputs of the backward, by name, from empty(shape, dtype)."""
        t, f32 = TORCH_DTYPE[self.dtype], torch.float32
        out = {"dx": empty((self.M, self.N), t), "dresidual": empty((self.M, self.N), t), "dweight": empty((self.N,), f32)}
        out["dnorm_weight"] = empty((self.N,), f32) if self.norm_weight is not None else None
        out["dgate"] = None
        if self.gate is not None:
            out["dgate"] = empty(tuple(self.gate.shape), f32 if self.gate_rows else t)
        return out

    @property
    def needs_sum(self):
        return self.norm_weight is not None or self.gate is not None
