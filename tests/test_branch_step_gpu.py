"""Dropout and the branch as a model uses them: a step of two tensor-parallel blocks behind an embedding that is split over
the ranks, with norms on both sides of each block, a gate per sample and one per column, and dropout, forward and backward,
against autograd in 64 bits; the same captured and replayed with a mask of its own each time.

Tolerance: every value is reached through at most ten fp32 products or normalisations in a row, each a sum of at most 256
terms; 10 * 256 roundings of 2^-24, all in one direction, are under 2^-12 of the norm of what is summed, and cancellation in
the residual's gradient at most doubles that: 2^-11 relative to the 2-norm."""
import pytest
import torch

from branch_checks import factor
from operator_checks import DEV, gen, randn, rank_sum

pytestmark = pytest.mark.gpu

W, S, L, N, K, EPS, P = 4, 3, 8, 256, 64, 1e-5, 0.25   # ranks, samples, their rows, hidden, a rank's inner width
M = S * L


@pytest.fixture(scope="module")
def car():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import rank_sum_reduce_gb300 as car

    return car


class Step:
    """x = drop(sum e_r); y0 = norm(x); block b: y -> sum_r y A_r B_r, normed, gated, dropped out and added."""

    def __init__(self, car, seed):
        g = gen(seed)
        weight = lambda: torch.rand(N, generator=g, device=DEV) + 0.5  # noqa: E731
        self.emb = [randn(g, (M, N), "fp32") for _ in range(W)]
        self.zero = torch.zeros(M, N, device=DEV)
        self.pre, self.post = [weight() for _ in range(3)], [weight() for _ in range(2)]
        self.gate = [randn(g, (S, N), "fp32", 0.7), randn(g, (N,), "fp32", 0.7)]
        self.A = [[randn(g, (N, K), "fp32", N**-0.5) for _ in range(W)] for _ in range(2)]
        self.B = [[randn(g, (K, N), "fp32", K**-0.5) for _ in range(W)] for _ in range(2)]
        self.dys = [randn(g, (M, N), "fp32", 0.1) for _ in range(W)]
        self.step = torch.zeros(1, dtype=torch.int64, device=DEV)
        self.seed, self.offsets = 5, [10**6, 2 * 10**6, 3 * 10**6]
        self.drops = [car.Dropout(P, self.seed, o, offset_dev=self.step) for o in self.offsets]
        self.branches = [car.Branch(self.post[b], EPS, self.gate[b], gate_rows=S if b == 0 else 1, residual_scale=0.9,
                                    dropout=self.drops[1 + b]) for b in range(2)]
        self.c = car.Car(W, M, N, "fp32")
        new = lambda *s: torch.empty(*s, device=DEV)  # noqa: E731
        self.x, self.h, self.y, self.a = new(M, N), [new(M, N) for _ in range(3)], [new(M, N) for _ in range(3)], \
            [new(M, N) for _ in range(2)]
        self.dx, self.dh = [new(M, N) for _ in range(2)], [new(M, N) for _ in range(3)]
        self.demb = new(M, N)
        self.dpre, self.dpost = [new(N) for _ in range(3)], [new(N) for _ in range(2)]
        self.dgate = [new(S, N), new(1, N)]

    def run(self):
        c = self.c
        c.reduce_dropout(self.emb, self.drops[0], self.x)
        c1 = self.one
        c1.reduce_residual_rmsnorm([self.zero], self.x, self.pre[0], EPS, self.h[0], self.y[0])
        self.z = []
        for b in range(2):
            z = [self.y[b] @ a for a in self.A[b]]
            self.z.append(z)
            c.reduce_branch_residual_rmsnorm([v @ w for v, w in zip(z, self.B[b])], self.branches[b], self.h[b], self.pre[b + 1],
                                             EPS, self.h[b + 1], self.y[b + 1], ar_out=self.a[b])
        # the loss is the sum of y2 times every rank's dys
        dys, dres = self.dys, None
        for b in (1, 0):
            c.reduce_branch_residual_rmsnorm_backward(dys, self.branches[b], self.a[b], self.h[b + 1], self.pre[b + 1], EPS, dres,
                                                      self.dx[b], self.dh[b], self.dpre[b + 1], self.dpost[b], self.dgate[b])
            dys, dres = [self.dx[b] @ w.T @ a.T for a, w in zip(self.A[b], self.B[b])], self.dh[b]
        c.reduce_residual_rmsnorm_backward(dys, self.h[0], self.pre[0], EPS, dres, self.dh[2], self.dpre[0])
        c1.reduce_dropout([self.dh[2]], self.drops[0], self.demb)

    def check(self):
        k = int(self.step)
        f = [factor(M, N, P, self.seed, o + k) for o in self.offsets]
        leaves = {n: [t.double().requires_grad_() for t in getattr(self, n)] for n in ("emb", "pre", "post", "gate")}
        norm = lambda v, w: v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * w  # noqa: E731
        h = sum(leaves["emb"]) * f[0]
        y = norm(h, leaves["pre"][0])
        for b in range(2):
            a = sum(y @ p.double() @ q.double() for p, q in zip(self.A[b], self.B[b]))
            g = leaves["gate"][b]
            g = g.repeat_interleave(L, 0) if b == 0 else g
            h = 0.9 * h + norm(a, leaves["post"][b]) * g * f[1 + b]
            y = norm(h, leaves["pre"][b + 1])
        (y * rank_sum(self.dys).double()).sum().backward()
        near = lambda u, v: float((u.double() - v).norm()) <= 2.0**-11 * float(v.norm())  # noqa: E731
        assert near(self.y[2], y.detach())
        for got, want in ((self.dpre, leaves["pre"]), (self.dpost, leaves["post"])):
            assert all(near(u, v.grad) for u, v in zip(got, want))
        assert near(self.dgate[0], leaves["gate"][0].grad) and near(self.dgate[1][0], leaves["gate"][1].grad)
        assert all(near(self.demb, e.grad) for e in leaves["emb"])   # every rank's embedding has the same gradient

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.c.close()
        self.one.close()


def make(car, seed):
    s = Step(car, seed)
    s.one = car.Car(1, M, N, "fp32")
    return s


def test_training_step_matches_autograd(car):
    with make(car, 3) as s:
        for _ in range(2):
            s.run()
            s.c.sync()
            s.check()
            s.step.add_(1)


def test_captured_step_has_a_new_mask_at_every_replay(car):
    with make(car, 4) as s:
        s.run()   # libraries of the products, outside the capture
        s.c.sync()
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            s.step.add_(1)
            s.run()
        last = None
        for _ in range(3):
            graph.replay()
            s.c.sync()
            s.check()
            assert last is None or not torch.equal(last, s.y[2])
            last = s.y[2].clone()
        del graph
