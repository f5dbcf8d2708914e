"""Backward of the fused op (car_reduce_residual_rmsnorm_backward) against its formula in 64 bits, against autograd of
the forward's definition, and against differences.

Tolerances (see operator_checks): with a = rms g w, b = rms u m and d the skip gradient, dx loses DELTA of each of
|a| and |d| and, since m is a mean of terms that may cancel, DELTA of rms |u| mean|g w u| for b, twice for the two sums
that enter it; plus its rounding.  dweight sums at most 14 rows in a register, 16 teams of a CTA, 19 partials in a
thread and 32 threads' sums: under 100 roundings of 2^-24, with those of g u under 2^-17 of sum |g u|."""
import pytest
import torch

from operator_checks import DELTA, DEV, TINY, TORCH_DTYPE, Guarded, assert_within, gen, half, randn, rank_sum

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def car():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import rank_sum_reduce_gb300 as car

    return car


def make(W, M, N, dtype, seed):
    g = gen(seed)
    dys = [randn(g, (M, N), dtype, 0.1) for _ in range(W)]
    h = randn(g, (M, N), dtype, 1.5)
    w = (torch.rand(N, generator=g, device=DEV) + 0.5).to(TORCH_DTYPE[dtype])
    return dys, h, w, randn(g, (M, N), dtype, 0.2)


def formula(dys, h, w, eps, dres):
    """(dx, bound without rounding, dweight, its bound) in 64 bits."""
    g, h, w = rank_sum(dys).double(), h.double(), w.double()
    r = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    u = h * r
    gwu = g * w * u
    m = gwu.mean(1, keepdim=True)
    d = torch.zeros_like(h) if dres is None else dres.double()
    dx = r * (g * w - u * m) + d
    bound = DELTA * ((r * g * w).abs() + d.abs() + 2 * (r * u).abs() * gwu.abs().mean(1, keepdim=True) + (r * u * m).abs())
    return dx, bound, (g * u).sum(0), 2.0**-17 * (g * u).abs().sum(0)


def check(dx, dw, dys, h, w, eps, dres, dtype):
    want, bound, want_dw, bound_dw = formula(dys, h, w, eps, dres)
    assert_within(dx, want, half(dtype) * want.abs() + (1 + half(dtype)) * bound + TINY[dtype], "dx")
    if dw is not None:
        assert_within(dw, want_dw, bound_dw, "dweight")


CASES = [
    # one CTA per row, two vectors per thread, rows split over 4 and 8 CTAs, many rows per CTA, the longest rows
    (1, 1, 8, "bf16"), (1, 2000, 40, "bf16"), (2, 1, 2048, "bf16"), (2, 37, 2056, "bf16"), (3, 7, 1000, "fp16"),
    (4, 300, 2056, "bf16"), (4, 160, 8192, "bf16"), (8, 1, 8192, "bf16"), (8, 24, 8200, "bf16"), (8, 700, 4104, "fp16"),
    (16, 2, 4100, "fp32"), (16, 9, 1544, "bf16"), (5, 2, 32768, "bf16"), (2, 4, 16384, "fp32"), (1, 33, 4, "fp32"),
    (4, 400, 4096, "fp32"), (8, 600, 132, "fp32"), (8, 400, 8192, "bf16"), (4, 500, 5000, "fp16"), (1, 700, 16384, "bf16"),
    (1, 600, 4096, "bf16"), (6, 200, 8200, "bf16"), (2, 330, 32768, "fp16"), (16, 170, 4224, "fp32"), (8, 310, 16384, "bf16"),
    # the pipeline kernel with four and eight vectors per thread, and with several teams whose last tile is not full
    (3, 401, 10000, "bf16"), (1, 311, 8192, "fp32"), (6, 230, 16384, "fp32"), (5, 197, 16384, "fp16"), (1, 1301, 1024, "bf16"),
    (3, 1001, 2056, "fp16"), (2, 901, 1000, "fp32"),
    # three vectors per thread
    (8, 401, 6144, "bf16"), (4, 331, 10488, "fp16"), (1, 311, 11072, "bf16"), (16, 307, 4656, "fp32"), (1, 1231, 12800, "fp32"),
    # four to eight, rows of more than 24 KB
    (8, 333, 13000, "bf16"), (1, 111, 9000, "fp32"), (8, 203, 10004, "fp32"), (2, 167, 11004, "fp32"), (6, 95, 12288, "fp32"),
    (4, 161, 13004, "fp32"), (1, 1301, 15000, "fp32"), (3, 91, 16384, "fp32"),
    # partials of several CTAs per SM, and more columns than blocks of 32 cover
    (2, 3001, 264, "fp16"), (8, 170, 4872, "bf16"),
]


@pytest.mark.parametrize("W,M,N,dtype", CASES)
@pytest.mark.parametrize("skip", [True, False])
def test_matches_formula(car, W, M, N, dtype, skip):
    dys, h, w, dres = make(W, M, N, dtype, seed=W * 1000 + M + N)
    dres = dres if skip else None
    out = Guarded()
    dx, dw = out.empty((M, N), TORCH_DTYPE[dtype]), out.empty((N,), torch.float32)
    with car.Car(W, M, N, dtype) as c:
        ws = out.empty((c.backward_workspace_bytes,), torch.uint8)
        c.reduce_residual_rmsnorm_backward(dys, h, w, 1e-6, dres, dx, dw, workspace=ws)
        c.sync()
        check(dx, dw, dys, h, w, 1e-6, dres, dtype)
        first = dx.clone(), dw.clone()
        c.reduce_residual_rmsnorm_backward(dys, h, w, 1e-6, dres, dx, dw)   # its own workspace; the same bits
        c.sync()
        assert torch.equal(dx, first[0]) and torch.equal(dw, first[1])
        dw.fill_(7.0)
        dx.fill_(7.0)
        c.reduce_residual_rmsnorm_backward(dys, h, w, 1e-6, dres, dx)       # no weight gradient
        c.sync()
        assert torch.equal(dx, first[0]) and (dw == 7.0).all()
    out.check()


@pytest.mark.parametrize("alias", ["dnorm", "h", "dres"])
@pytest.mark.parametrize("W,M,N", [(4, 37, 1032), (4, 400, 8192), (8, 2, 8192)])
def test_dx_may_replace_an_input(car, alias, W, M, N):
    dys, h, w, dres = make(W, M, N, "bf16", seed=3)
    keep = [d.clone() for d in dys], h.clone(), dres.clone()
    dx = {"dnorm": dys[1], "h": h, "dres": dres}[alias]
    dw = torch.empty(N, device=DEV)
    with car.Car(W, M, N, "bf16") as c:
        c.reduce_residual_rmsnorm_backward(dys, h, w, 1e-6, dres, dx, dw)
        c.sync()
    check(dx, dw, keep[0], keep[1], w, 1e-6, keep[2], "bf16")


def loss(xs, res, w, eps, dy, dro):
    h = sum(xs) + res
    return (h * torch.rsqrt((h * h).mean(1, keepdim=True) + eps) * w * dy).sum() + (h * dro).sum()


def test_matches_autograd_and_differences(car):
    """fp32, eps large enough to matter: autograd of the forward in 64 bits, and central differences of its loss along
    random directions.  A step of 1e-4 leaves 1e-8 of the third derivative, far below the fp32 bound."""
    W, M, N, eps = 3, 5, 260, 0.3
    g = gen(4)
    xs, res = [randn(g, (M, N), "fp32", 0.5).double() for _ in range(W)], randn(g, (M, N), "fp32").double()
    dys, _, w, dro = make(W, M, N, "fp32", seed=9)
    h32 = (sum(xs) + res).float()
    res = h32.double() - sum(xs)  # so that the stored h is the forward's
    dx, dw = torch.empty(M, N, device=DEV), torch.empty(N, device=DEV)
    with car.Car(W, M, N, "fp32") as c:
        c.reduce_residual_rmsnorm_backward(dys, h32, w, eps, dro, dx, dw)
        c.sync()
    leaves = [t.clone().requires_grad_() for t in (*xs, res, w.double())]
    dy, dr = rank_sum(dys).double(), dro.double()
    loss(leaves[:W], leaves[W], leaves[W + 1], eps, dy, dr).backward()
    _, bound, _, bound_dw = formula(dys, h32, w, eps, dro)
    for leaf in leaves[:W + 1]:   # the residual and every rank have the same gradient
        assert_within(dx, leaf.grad, bound + half("fp32") * leaf.grad.abs(), "dx against autograd")
    assert_within(dw, leaves[W + 1].grad, bound_dw, "dweight against autograd")
    for k in range(4):
        vx, vw = randn(g, (M, N), "fp32").double(), randn(g, (N,), "fp32").double()
        e = 1e-4
        up = loss([xs[0] + e * vx, *xs[1:]], res, w.double() + e * vw, eps, dy, dr)
        dn = loss([xs[0] - e * vx, *xs[1:]], res, w.double() - e * vw, eps, dy, dr)
        got = (dx.double() * vx).sum() + (dw.double() * vw).sum()
        room = (bound * vx.abs()).sum() + (bound_dw * vw.abs()).sum() + half("fp32") * (dx.double() * vx).abs().sum()
        assert abs(got - (up - dn) / (2 * e)) <= room + 1e-6 * abs(got)


def test_zero_rows_and_nan(car):
    W, M, N = 2, 6, 512
    dys, h, w, dres = make(W, M, N, "bf16", seed=6)
    h[0] = 0                      # u = 0: dx = g w / sqrt(eps) + dres, nothing for dweight
    h[3, 5] = float("nan")
    dx, dw = torch.empty_like(h), torch.empty(N, device=DEV)
    with car.Car(W, M, N, "bf16") as c:
        c.reduce_residual_rmsnorm_backward(dys, h, w, 1e-4, dres, dx, dw)
        c.sync()
    assert dx[3].isnan().all() and dw.isnan().all()
    rest = [0, 1, 2, 4, 5]
    check(dx[rest], None, [d[rest] for d in dys], h[rest], w, 1e-4, dres[rest], "bf16")


def test_captured_with_its_own_workspace(car):
    W, M, N = 4, 300, 2056
    dys, h, w, dres = make(W, M, N, "bf16", seed=12)
    dx, dw = torch.empty_like(h), torch.empty(N, device=DEV)
    with car.Car(W, M, N, "bf16") as c:
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            c.reduce_residual_rmsnorm_backward(dys, h, w, 1e-6, dres, dx, dw)
        for seed in (13, 14):
            new = make(W, M, N, "bf16", seed=seed)
            for a, b in zip(dys + [h, w, dres], new[0] + list(new[1:])):
                a.copy_(b)
            graph.replay()
            c.sync()
            check(dx, dw, dys, h, w, 1e-6, dres, "bf16")
        del graph


def test_two_streams_at_once_with_two_workspaces(car):
    W, M, N = 2, 500, 4096
    sets = [make(W, M, N, "bf16", seed=31 + k) for k in range(2)]
    outs = [(torch.empty(M, N, device=DEV).bfloat16(), torch.empty(N, device=DEV)) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    with car.Car(W, M, N, "bf16") as c:
        ws = [torch.empty(c.backward_workspace_bytes, dtype=torch.uint8, device=DEV) for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(5):
            for (dys, h, w, dres), (dx, dw), s, b in zip(sets, outs, streams, ws):
                c.reduce_residual_rmsnorm_backward(dys, h, w, 1e-6, dres, dx, dw, workspace=b, stream=s)
        torch.cuda.synchronize()
        for (dys, h, w, dres), (dx, dw) in zip(sets, outs):
            check(dx, dw, dys, h, w, 1e-6, dres, "bf16")
        with pytest.raises(ValueError):  # no workspace to be had for a stream that is not the current one
            c.reduce_residual_rmsnorm_backward(*sets[0][:3], 1e-6, sets[0][3], *outs[0], stream=streams[0])


def test_refusals(car):
    W, M, N = 2, 400, 64
    dys, h, w, dres = make(W, M, N, "bf16", seed=1)
    dx, dw = torch.empty_like(h), torch.empty(N, device=DEV)
    with car.Car(W, M, N, "bf16") as c:
        ws = torch.empty(c.backward_workspace_bytes, dtype=torch.uint8, device=DEV)
        P = lambda t: t.data_ptr()  # noqa: E731
        ok = dict(h=c.h, dnorm=[P(d) for d in dys], residual_out=P(h), weight=P(w), eps=1e-6, dresidual_out=P(dres),
                  dx=P(dx), dweight=P(dw), workspace=P(ws), stream=0)
        call = lambda **k: car.car_reduce_residual_rmsnorm_backward(**{**ok, **k})  # noqa: E731
        for k in (dict(eps=-1.0), dict(eps=float("inf")), dict(dnorm=None), dict(residual_out=None), dict(weight=None),
                  dict(dx=None), dict(workspace=None)):
            assert call(**k) == car.CAR_ERR_ARG, k
        for k in (dict(dx=P(dx) + 2), dict(dweight=P(dw) + 4), dict(workspace=P(ws) + 8), dict(dresidual_out=P(dres) + 2)):
            assert call(**k) == car.CAR_ERR_ALIGN, k
        assert call(workspace=None, dweight=None) == car.CAR_OK
        with pytest.raises(ValueError):
            c.reduce_residual_rmsnorm_backward(dys, h, w, 1e-6, dres, dx, dw, workspace=ws[:-1])
        with pytest.raises(ValueError):
            c.reduce_residual_rmsnorm_backward(dys, h, w, 1e-6, dres, dx, dw[:-1])
        c.sync()
    assert car.car_backward_workspace_bytes(None) == 0
