"""The operators next to the rank sum, together and at their edges: a training step of a small tensor-parallel,
data-parallel model against autograd in 64 bits, the same captured and replayed, rows and tensors past 32-bit offsets,
waits that run out, streams.

Tolerance of the training step: every value is reached through at most eight fp32 products or normalisations in a row,
each a sum of at most 256 terms; 8 * 256 roundings of 2^-24, all in one direction, are 2^-13 of the norm of what is
summed, and cancellation in the residual's gradient at most doubles that: 2^-12 relative to the 2-norm."""
import math

import pytest
import torch

from operator_checks import DELTA, DEV, Guarded, assert_within, gen, half, randn, rank_sum

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def car():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import rank_sum_reduce_gb300 as car

    return car


# ---------------------------------------------------------------------------
# a training step
# ---------------------------------------------------------------------------
W, M, N, K, EPS = 4, 24, 256, 64, 1e-5   # ranks of the tensor-parallel group, tokens, hidden, a rank's inner width
REPLICAS = 2                              # data-parallel replicas


class Step:
    """norm(sum x_r + res) -> each rank's two products -> norm(sum o_r + h1), in fp32, and its gradients."""

    def __init__(self, car, seed):
        g = gen(seed)
        self.w1, self.w2 = (torch.rand(N, generator=g, device=DEV) + 0.5 for _ in range(2))
        self.B = [randn(g, (N, K), "fp32", N**-0.5) for _ in range(W)]
        self.C = [randn(g, (K, N), "fp32", K**-0.5) for _ in range(W)]
        self.data = [self.draw(g) for _ in range(REPLICAS)]
        self.car = car.Car(W, M, N, "fp32")
        self.h = [[torch.empty(M, N, device=DEV) for _ in range(2)] for _ in range(REPLICAS)]
        self.y = [[torch.empty(M, N, device=DEV) for _ in range(2)] for _ in range(REPLICAS)]
        self.dx = [[torch.empty(M, N, device=DEV) for _ in range(2)] for _ in range(REPLICAS)]
        like = [self.w1, self.w2, *self.B, *self.C]
        self.grads = [[torch.empty_like(t) for t in like] for _ in range(REPLICAS)]
        self.total = [torch.empty_like(t) for t in like]
        self.norm = torch.empty(1, device=DEV)
        self.q = torch.empty(M, N, dtype=torch.float8_e4m3fn, device=DEV)
        self.s = torch.empty(M, 1, device=DEV)
        self.clip = car.Grads(self.grads, self.total)

    @staticmethod
    def draw(g):
        xs = [randn(g, (M, N), "fp32", 0.5) for _ in range(W)]
        return xs, randn(g, (M, N), "fp32"), [randn(g, (M, N), "fp32", 0.1) for _ in range(W)]

    def run(self, max_norm):
        c = self.car
        for r, (xs, res, dys) in enumerate(self.data):
            (h1, h2), (y1, y2), (dx1, dx2), grads = self.h[r], self.y[r], self.dx[r], self.grads[r]
            dw1, dw2, dB, dC = grads[0], grads[1], grads[2:2 + W], grads[2 + W:]
            c.reduce_residual_rmsnorm(xs, res, self.w1, EPS, h1, y1)
            z = [y1 @ b for b in self.B]
            c.reduce_residual_rmsnorm([a @ b for a, b in zip(z, self.C)], h1, self.w2, EPS, h2, y2)
            # the loss is the sum of y2 times every rank's dys; h2 goes nowhere else
            c.reduce_residual_rmsnorm_backward(dys, h2, self.w2, EPS, None, dx2, dw2)
            dy1 = []
            for k in range(W):
                dz = dx2 @ self.C[k].T
                dC[k].copy_(z[k].T @ dx2)
                dB[k].copy_(y1.T @ dz)
                dy1.append(dz @ self.B[k].T)
            c.reduce_residual_rmsnorm_backward(dy1, h1, self.w1, EPS, dx2, dx1, dw1)
        # what a server would take of the last replica's first norm
        xs, res, _ = self.data[-1]
        c.reduce_residual_rmsnorm_quant(xs, res, self.w1, EPS, "row", self.h[-1][0], self.q, self.s)
        self.clip.reduce_clip(1.0 / REPLICAS, max_norm, self.norm)

    def check(self, max_norm):
        total, dxs = None, []
        for xs, res, dys in self.data:
            leaves = [t.double().requires_grad_() for t in (self.w1, self.w2, *self.B, *self.C, res, *xs)]
            w1, w2, B, C, x = leaves[0], leaves[1], leaves[2:2 + W], leaves[2 + W:2 + 2 * W], leaves[2 + 2 * W:]
            norm = lambda h, w: h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * w  # noqa: E731
            h1 = sum(x)
            y1 = norm(h1, w1)
            h2 = sum(y1 @ b @ c for b, c in zip(B, C)) + h1
            (norm(h2, w2) * sum(d.double() for d in dys)).sum().backward()
            got = [t.grad for t in leaves[:2 + 2 * W]]
            dxs.append([t.grad for t in leaves[2 + 2 * W:]])
            total = got if total is None else [a + b for a, b in zip(total, got)]
            y_last = y1.detach()
        total = [t / REPLICAS for t in total]
        size = math.sqrt(sum(float((t * t).sum()) for t in total))
        near = lambda a, b: float((a.double() - b).norm()) <= 2.0**-12 * float(b.norm())  # noqa: E731
        assert abs(self.norm.item() - size) <= 2.0**-12 * size
        factor = min(1.0, max_norm / (size + 1e-6))
        for got, want in zip(self.total, total):
            assert near(got, want * factor)
        for r in range(REPLICAS):
            for want in dxs[r]:   # the residual's gradient and every rank's are the same
                assert near(self.dx[r][0], want)
        v = y_last / self.s.double()
        assert (v.abs().amax(1) <= 448 * (1 + 2.0**-12)).all()
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0**-6)))) / 8
        assert_within(self.q, v.clamp(-448, 448), step / 2 + 2.0**-12 * v.abs() + 2.0**-12, "q")


@pytest.mark.parametrize("max_norm", [1e-2, 1e9])
def test_training_step_eager_and_captured(car, max_norm):
    step = Step(car, seed=3)
    step.run(max_norm)
    torch.cuda.synchronize()
    step.check(max_norm)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        step.run(max_norm)
    g = gen(77)
    for xs, res, dys in step.data:
        nx, nr, nd = Step.draw(g)
        for a, b in zip([*xs, res, *dys], [*nx, nr, *nd]):
            a.copy_(b)
    graph.replay()
    step.car.sync()
    torch.cuda.synchronize()
    step.check(max_norm)
    first = [t.clone() for t in (*step.total, step.norm, step.dx[0][0], step.s)]
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (*step.total, step.norm, step.dx[0][0], step.s)))
    del graph
    step.clip.close()
    step.car.close()


# ---------------------------------------------------------------------------
# offsets past 32 bits
# ---------------------------------------------------------------------------
def test_quant_rows_past_32_bit_offsets(car):
    M, N = 280_007, 8192      # 2.3e9 elements: codes past 2^31 bytes, 16-bit rows past 2^32
    x = torch.empty(M, N, dtype=torch.bfloat16, device=DEV).normal_(generator=gen(1))
    res = torch.empty(M, N, dtype=torch.bfloat16, device=DEV).normal_(generator=gen(2))
    w = (torch.rand(N, generator=gen(3), device=DEV) + 0.5).bfloat16()
    ro, q = torch.empty_like(res), torch.empty(M, N, dtype=torch.float8_e4m3fn, device=DEV)
    with car.Car(1, M, N, "bf16") as c:
        s = torch.empty(c.quant_scales_shape("group128"), device=DEV)
        c.reduce_residual_rmsnorm_quant([x], res, w, 1e-6, "group128", ro, q, s)
        c.sync()
    for rows in (slice(0, 40), slice(131_050, 131_100), slice(262_130, 262_160), slice(M - 40, M)):
        h = x[rows].float() + res[rows].float()
        assert torch.equal(ro[rows], h.bfloat16())
        d = h.double()
        y = d * w.double() / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-6)
        amax = y.abs().reshape(len(y), -1, 128).amax(2)
        assert_within(s[rows], amax / 448, DELTA * amax / 448, "scales")
        v = (y / s[rows].double().repeat_interleave(128, 1)).clamp(-448, 448)
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0**-6)))) / 8
        assert_within(q[rows], v, step / 2 + 2 * DELTA * v.abs(), "q")


def test_backward_rows_past_32_bit_offsets(car):
    M, N = 280_007, 8192
    dy = torch.empty(M, N, dtype=torch.bfloat16, device=DEV).normal_(generator=gen(4))
    h = torch.empty(M, N, dtype=torch.bfloat16, device=DEV).normal_(generator=gen(5))
    w = (torch.rand(N, generator=gen(6), device=DEV) + 0.5).bfloat16()
    dx, dw = torch.empty_like(h), torch.empty(N, device=DEV)
    with car.Car(1, M, N, "bf16") as c:
        c.reduce_residual_rmsnorm_backward([dy], h, w, 1e-6, None, dx, dw)
        c.sync()
    want_dw, room = torch.zeros(N, dtype=torch.float64, device=DEV), torch.zeros(N, dtype=torch.float64, device=DEV)
    for at in range(0, M, 20_000):
        rows = slice(at, min(M, at + 20_000))
        hd, g = h[rows].double(), dy[rows].double()
        u = hd / torch.sqrt((hd * hd).mean(1, keepdim=True) + 1e-6)
        want_dw += (g * u).sum(0)
        room += (g * u).abs().sum(0)
        if at in (0, 120_000, 260_000) or rows.stop == M:
            r = 1 / torch.sqrt((hd * hd).mean(1, keepdim=True) + 1e-6)
            gwu = g * w.double() * u
            m = gwu.mean(1, keepdim=True)
            want = r * (g * w.double() - u * m)
            bound = DELTA * ((r * g * w.double()).abs() + 3 * (r * u).abs() * gwu.abs().mean(1, keepdim=True))
            assert_within(dx[rows], want, half("bf16") * want.abs() + 1.01 * bound, f"dx from row {at}")
    # a CTA's registers take M / 152 rows in a row
    assert_within(dw, want_dw, (M / 148 + 100) * 2.0**-24 * room + 2.0**-18 * room, "dweight")


def test_one_tensor_of_more_than_4_gb(car):
    n = (1 << 31) + 100_001
    x = torch.empty(n, dtype=torch.bfloat16, device=DEV).normal_(generator=gen(7))
    x[-3] = 3000.0
    out, nb = torch.empty_like(x), torch.empty(1, device=DEV)
    with car.Grads([[x]], [out]) as g:
        g.reduce_clip(0.5, 1.0, nb)
        torch.cuda.synchronize()
    size = 0.5 * math.sqrt(sum(float((p.double() ** 2).sum()) for p in x.split(1 << 28)))
    assert abs(nb.item() - size) <= 2.0**-18 * size
    for part in (slice(0, 1000), slice((1 << 30) - 500, (1 << 30) + 500), slice((1 << 31) - 500, (1 << 31) + 500),
                 slice(n - 1000, n)):
        want = x[part].double() * 0.5 / (size + 1e-6)
        assert_within(out[part], want, (half("bf16") + 2.0**-18) * want.abs() + 2.0**-134, "values")


# ---------------------------------------------------------------------------
# edges
# ---------------------------------------------------------------------------
def test_gradients_without_a_single_value(car):
    e = torch.empty(0, device=DEV)
    nb, s = torch.full((1,), 5.0, device=DEV), torch.full((1,), 5.0, dtype=torch.float64, device=DEV)
    with car.Grads([[e, e], [e, e]], [e, e]) as g:
        g.reduce_clip(1.0, 1.0, nb)
        g.reduce(1.0, s)
        torch.cuda.synchronize()
    assert nb.item() == 0 and s.item() == 0


@pytest.mark.parametrize("kind", ["row", "mx32"])
@pytest.mark.parametrize("cta", [0, 3])
def test_late_partial_of_a_quantised_row(car, kind, cta):
    """The bounded wait made to run out (see tests/test_wait_timeout_gpu.py): NaN codes for the columns of the threads
    that gave up, everything else right, the next call clean."""
    W, M, N, row = 8, 4, 8192, 2   # clusters of 8 CTAs, 1024 columns each
    g = gen(9)
    xs, res = [randn(g, (M, N), "bf16") for _ in range(W)], randn(g, (M, N), "bf16")
    w = (torch.rand(N, generator=g, device=DEV) + 0.5).bfloat16()
    outs = [(torch.empty_like(res), torch.empty(M, N, dtype=torch.float8_e4m3fn, device=DEV)) for _ in range(2)]
    stream = torch.cuda.current_stream().cuda_stream
    with car.Car(W, M, N, "bf16") as c:
        ss = [torch.empty(c.quant_scales_shape(kind), device=DEV, dtype=torch.uint8 if kind == "mx32" else torch.float32)
              for _ in range(2)]
        torch.cuda.synchronize()
        assert car.car_test_delay_partial(c.h, 50_000, cta, row, 2_000_000) == car.CAR_OK
        c.reduce_residual_rmsnorm_quant(xs, res, w, 1e-6, kind, outs[0][0], outs[0][1], ss[0])
        assert car.car_sync(c.h, stream) == car.CAR_ERR_TIMEOUT
        assert car.car_test_delay_partial(c.h, 0, -1, 0, 0) == car.CAR_OK
        c.reduce_residual_rmsnorm_quant(xs, res, w, 1e-6, kind, outs[1][0], outs[1][1], ss[1])
        assert car.car_sync(c.h, stream) == car.CAR_OK
    torch.cuda.synchronize()
    h = rank_sum(xs) + res.float()
    assert all(torch.equal(ro, h.bfloat16()) for ro, _ in outs)
    late, right = outs[0][1].float(), outs[1][1].float()
    assert right.isfinite().all()
    mine = torch.zeros(N, dtype=torch.bool, device=DEV)
    mine[cta * 1024:(cta + 1) * 1024] = True
    assert torch.equal(late[row][mine], right[row][mine]) and late[row][~mine].isnan().all()
    rest = [r for r in range(M) if r != row]
    assert torch.equal(late[rest], right[rest]) and torch.equal(ss[0][rest], ss[1][rest])
    if kind == "row":   # the scale is the first CTA's to write
        assert ss[0][row].isnan().all() if cta else torch.equal(ss[0][row], ss[1][row])
    else:
        lost = ~mine[::32]
        assert (ss[0][row][lost] == 255).all() and torch.equal(ss[0][row][~lost], ss[1][row][~lost])


def test_late_partial_of_a_backward_row(car):
    W, M, N, row, cta = 8, 4, 8192, 1, 5
    g = gen(10)
    dys, h = [randn(g, (M, N), "bf16", 0.1) for _ in range(W)], randn(g, (M, N), "bf16")
    w = (torch.rand(N, generator=g, device=DEV) + 0.5).bfloat16()
    outs = [(torch.empty_like(h), torch.empty(N, device=DEV)) for _ in range(2)]
    stream = torch.cuda.current_stream().cuda_stream
    with car.Car(W, M, N, "bf16") as c:
        assert car.car_test_delay_partial(c.h, 50_000, cta, row, 2_000_000) == car.CAR_OK
        c.reduce_residual_rmsnorm_backward(dys, h, w, 1e-6, None, *outs[0])
        assert car.car_sync(c.h, stream) == car.CAR_ERR_TIMEOUT
        assert car.car_test_delay_partial(c.h, 0, -1, 0, 0) == car.CAR_OK
        c.reduce_residual_rmsnorm_backward(dys, h, w, 1e-6, None, *outs[1])
        assert car.car_sync(c.h, stream) == car.CAR_OK
    (late, late_dw), (right, right_dw) = outs
    assert right.isfinite().all() and right_dw.isfinite().all()
    mine = torch.zeros(N, dtype=torch.bool, device=DEV)
    mine[cta * 1024:(cta + 1) * 1024] = True
    assert torch.equal(late[row][mine], right[row][mine]) and late[row][~mine].isnan().all()
    rest = [r for r in range(M) if r != row]
    assert torch.equal(late[rest], right[rest])
    assert late_dw[~mine].isnan().all() and torch.equal(late_dw[mine], right_dw[mine])


def test_quantised_calls_of_one_handle_on_two_streams(car):
    W, M, N = 2, 900, 2048
    sets = []
    for k in range(2):
        g = gen(50 + k)
        sets.append(([randn(g, (M, N), "bf16") for _ in range(W)], randn(g, (M, N), "bf16"), torch.ones(N, device=DEV).bfloat16()))
    out = Guarded()
    with car.Car(W, M, N, "bf16") as c:
        res = [(out.empty((M, N), torch.bfloat16), out.empty((M, N), torch.float8_e4m3fn), out.empty((M, 1), torch.float32))
               for _ in range(2)]
        for (xs, r, w), o in zip(sets, res):
            c.reduce_residual_rmsnorm_quant(xs, r, w, 1e-6, "row", *o)
        torch.cuda.synchronize()
        want = [[t.clone() for t in o] for o in res]
        streams = [torch.cuda.Stream() for _ in range(2)]
        for _ in range(8):
            for (xs, r, w), o, s in zip(sets, res, streams):
                c.reduce_residual_rmsnorm_quant(xs, r, w, 1e-6, "row", *o, stream=s)
        torch.cuda.synchronize()
    for o, v in zip(res, want):
        assert torch.equal(o[0], v[0]) and torch.equal(o[1].view(torch.uint8), v[1].view(torch.uint8)) and torch.equal(o[2], v[2])
    out.check()


def test_handles_of_different_shapes_share_the_kernels(car):
    """Handles whose pipelines run the same kernel instances with other ring sizes, made in every order: each still
    launches after the others exist."""
    shapes = [(8, 512, 8192, "bf16"), (1, 2500, 4096, "bf16"), (4, 700, 6144, "bf16"), (2, 2600, 2048, "bf16")]
    for order in (shapes, shapes[::-1]):
        cs = [car.Car(*s) for s in order]
        for c, (W, M, N, _) in zip(cs, order):
            g = gen(W + M)
            xs, h = [randn(g, (M, N), "bf16") for _ in range(W)], randn(g, (M, N), "bf16")
            w, ro, q = torch.ones(N, device=DEV).bfloat16(), torch.empty_like(h), torch.empty(M, N, dtype=torch.uint8, device=DEV)
            c.reduce_residual_rmsnorm_quant(xs, h, w, 1e-6, "row", ro, q, torch.empty(M, 1, device=DEV))
            c.reduce_residual_rmsnorm_backward(xs, h, w, 1e-6, None, torch.empty_like(h), torch.empty(N, device=DEV))
            c.sync()
            assert torch.equal(ro, (rank_sum(xs) + h.float()).bfloat16())
        for c in cs:
            c.close()


def test_plain_pipeline_handles_share_their_kernels(car):
    """The same for the fused op's pipeline: a handle with a smaller ring made later, or in between."""
    W, M = 8, 300
    big, small = car.Car(W, M, 8192, "bf16"), car.Car(W, M, 6144, "bf16")
    for c in (big, small, big):
        g = gen(c.N)
        xs, res = [randn(g, (M, c.N), "bf16") for _ in range(W)], randn(g, (M, c.N), "bf16")
        ro, no = torch.empty_like(res), torch.empty_like(res)
        c.tune_fused(car.CAR_FUSED_PIPELINE)
        small.tune_fused(car.CAR_FUSED_PIPELINE)
        c.reduce_residual_rmsnorm(xs, res, torch.ones(c.N, device=DEV).bfloat16(), 1e-6, ro, no)
        c.sync()
        assert torch.equal(ro, (rank_sum(xs) + res.float()).bfloat16())
    big.close()
    small.close()
