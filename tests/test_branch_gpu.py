"""A block's branch (car_reduce_branch_residual_rmsnorm and its backward) against the formulas in 64 bits, autograd and
differences; edges, aliases, streams, captures, refusals.  Tolerances: see branch_checks."""
import threading

import pytest
import torch

from branch_checks import Case, factor
from operator_checks import DELTA, DEV, TORCH_DTYPE, Guarded, assert_within, gen, half, randn, rank_sum

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def car():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import rank_sum_reduce_gb300 as car

    return car


def empty(shape, dtype):
    return torch.empty(shape, dtype=dtype, device=DEV)


def run_forward(c, k, branch, out, keep=True, **kw):
    t = TORCH_DTYPE[k.dtype]
    got = {"residual_out": out((k.M, k.N), t), "norm_out": out((k.M, k.N), t), "ar": out((k.M, k.N), t) if keep else None}
    c.reduce_branch_residual_rmsnorm(k.xs, branch, k.residual, k.weight, k.eps, got["residual_out"], got["norm_out"],
                                     ar_out=got["ar"], **kw)
    return got


def run_backward(c, k, branch, got, **kw):
    c.reduce_branch_residual_rmsnorm_backward(k.dys, branch, k.a if k.needs_sum else None, k.h, k.weight, k.eps, k.dres,
                                              got["dx"], got["dresidual"], got["dweight"], got["dnorm_weight"], got["dgate"],
                                              **kw)
    return got


# W, M, N, type, norm, gate rows (None: none; 0: a row for each), residual scale, p
CASES = [
    # one token, whole rows, rows split over 2, 4 and 8 CTAs, the longest rows
    (1, 1, 8, "bf16", True, None, 1.0, 0.0), (2, 1, 2048, "bf16", True, None, 1.0, 0.0), (1, 1, 4, "fp32", True, 1, 0.5, 0.1),
    (8, 24, 8192, "bf16", True, None, 1.0, 0.0), (8, 2, 8200, "fp16", True, 1, 1.0, 0.2), (4, 3, 16384, "fp32", True, 0, 2.0, 0.1),
    (5, 2, 32768, "bf16", True, 2, 1.0, 0.5), (3, 7, 1000, "fp16", False, None, 1.0, 0.3), (16, 9, 1544, "bf16", True, 3, -0.5, 0.0),
    (6, 1, 4100, "fp32", False, 0, 1.0, 0.0), (2, 37, 2056, "bf16", True, 37, 1.0, 0.1), (8, 12, 5000, "bf16", True, 4, 0.7, 0.0),
    # more rows than CTAs; gate rows that several CTAs share, that several CTAs cut, that lie whole in one
    (1, 2000, 40, "bf16", True, None, 1.0, 0.1), (1, 1333, 1160, "fp16", False, 31, 1.0, 0.0), (4, 1030, 520, "bf16", True, 5, 1.0, 0.1),
    (2, 1200, 264, "fp32", True, 400, 1.0, 0.0), (2, 900, 264, "bf16", False, 900, 1.25, 0.2), (4, 300, 2056, "bf16", True, 1, 0.0, 0.0),
    (16, 310, 520, "fp16", True, 0, 1.0, 0.1), (3, 500, 1032, "bf16", False, 0, 1.0, 0.0), (8, 700, 4104, "fp16", True, 7, 1.0, 0.0),
    # many rows
    (4, 160, 8192, "bf16", True, None, 1.0, 0.0), (4, 400, 4096, "fp32", True, 1, 0.75, 0.0), (8, 600, 132, "fp32", True, 2, 1.0, 0.1),
    (8, 400, 8192, "bf16", True, None, 1.0, 0.1), (4, 500, 5000, "fp16", False, 4, 1.0, 0.1), (1, 700, 16384, "bf16", True, None, 1.0, 0.0),
    (1, 600, 4096, "bf16", True, 6, 1.0, 0.1), (6, 200, 8200, "bf16", True, 0, 1.0, 0.0), (2, 330, 32768, "fp16", True, 1, 1.0, 0.1),
    (16, 170, 4224, "fp32", True, 17, 1.0, 0.0), (3, 401, 10000, "bf16", True, None, 1.0, 0.1), (1, 311, 8192, "fp32", True, 0, 1.0, 0.1),
    (1, 1301, 1024, "bf16", True, 1, 1.0, 0.0), (3, 1001, 2056, "fp16", True, 7, 1.0, 0.2), (2, 901, 1000, "fp32", False, 17, 1.0, 0.0),
    (8, 401, 6144, "bf16", True, 0, 1.0, 0.0), (4, 331, 10488, "fp16", True, 1, 1.0, 0.0), (1, 1231, 12800, "fp32", True, None, 1.0, 0.0),
    (8, 333, 13000, "bf16", True, 3, 1.0, 0.0), (2, 167, 11004, "fp32", True, None, 1.0, 0.1), (4, 161, 13004, "fp32", False, 7, 1.0, 0.0),
    (3, 182, 16384, "fp32", True, 2, 1.0, 0.0), (2, 3000, 264, "fp16", True, 1000, 1.0, 0.1), (1, 3001, 512, "bf16", False, None, 0.3, 0.5),
    (1, 2800, 2048, "fp16", True, 14, 1.0, 0.0),
    # three vectors per thread forward, clusters of two and four with each kind of gate, gate rows of few and of many rows
    (4, 320, 5120, "bf16", True, 1, 1.0, 0.0), (2, 480, 5128, "fp16", True, 4, 1.0, 0.1), (1, 460, 6144, "fp32", True, 0, 1.0, 0.0),
    (2, 200, 12296, "bf16", True, 0, 1.0, 0.1), (1, 156, 20488, "bf16", True, 2, 1.0, 0.0), (1, 155, 32768, "fp16", True, 155, 1.0, 0.0),
    (3, 154, 16384, "fp32", True, 7, 1.0, 0.1), (2, 2432, 1536, "bf16", True, 1216, 1.0, 0.0), (4, 1824, 648, "fp32", False, 912, 1.0, 0.2),
    (16, 640, 2064, "bf16", True, 5, 1.0, 0.1), (12, 310, 4104, "fp16", True, 1, 1.0, 0.0),
    # slices that leave the backward's ring room for less than two tiles
    (4, 400, 8192, "bf16", True, 4, 1.0, 0.1), (8, 320, 8192, "fp16", True, 0, 1.0, 0.1), (6, 200, 16384, "bf16", True, 0, 1.0, 0.1),
    (4, 200, 16384, "fp16", True, 2, 1.0, 0.1), (4, 170, 16384, "bf16", True, None, 1.0, 0.1), (16, 180, 16384, "fp16", True, 0, 1.0, 0.0),
    (5, 330, 7000, "bf16", True, 11, 1.0, 0.0), (16, 156, 32768, "bf16", True, 1, 1.0, 0.1),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_forward_matches_formula(car, case):
    k = Case(*case)
    out = Guarded()
    with car.Car(*case[:4]) as c:
        b = k.branch(car)
        got = run_forward(c, k, b, out.empty)
        c.sync()
        k.check_forward(got)
        again = run_forward(c, k, b, out.empty, keep=False)   # without the sum; the same bits
        c.sync()
        for name in ("residual_out", "norm_out"):
            assert torch.equal(got[name], again[name])
    out.check()


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_backward_matches_formula(car, case):
    k = Case(*case, skip=case[1] % 3 != 0)
    out = Guarded()
    with car.Car(*case[:4]) as c:
        b = k.branch(car)
        ws = out.empty((c.branch_workspace_bytes(b),), torch.uint8)
        got = run_backward(c, k, b, k.grads(out.empty), workspace=ws)
        c.sync()
        k.check_backward(got)
        again = run_backward(c, k, b, k.grads(out.empty))          # its own workspace; the same bits
        c.sync()
        assert all(t is None or torch.equal(t, again[name]) for name, t in got.items())
        only = out.empty((k.M, k.N), TORCH_DTYPE[k.dtype])          # dx alone
        ar = k.a if k.norm_weight is not None else None
        c.reduce_branch_residual_rmsnorm_backward(k.dys, b, ar, k.h, k.weight, k.eps, k.dres, only)
        c.sync()
        assert torch.equal(only, got["dx"])
    out.check()


def test_without_parts_it_is_the_fused_op(car):
    """residual_out and the sum bit for bit; norm_out within both calls' bounds."""
    for W, M, N, dtype in ((4, 33, 2056, "bf16"), (8, 300, 8192, "bf16"), (2, 5, 4100, "fp32"), (3, 700, 520, "fp16")):
        k = Case(W, M, N, dtype, norm=False)
        with car.Car(W, M, N, dtype) as c:
            got = run_forward(c, k, car.Branch(), empty)
            ro, no, ar = (torch.empty_like(k.residual) for _ in range(3))
            c.reduce_residual_rmsnorm(k.xs, k.residual, k.weight, k.eps, ro, no, ar)
            c.sync()
        assert torch.equal(got["residual_out"], ro) and torch.equal(got["ar"], ar)
        k.check_forward(got)


def test_a_branch_that_cancels_the_residual(car):
    """h is a few millionths of both terms of its sum: what is left is its own, not a difference of large sums."""
    W, M, N = 2, 40, 2048
    k = Case(W, M, N, "fp32", norm=False)
    k.xs = [torch.randn(M, N, device=DEV) * 100 for _ in range(W)]
    k.residual = -(rank_sum(k.xs)) + torch.randn(M, N, device=DEV) * 1e-3
    with car.Car(W, M, N, "fp32") as c:
        got = run_forward(c, k, k.branch(car), empty)
        c.sync()
    k.check_forward(got)


@pytest.mark.parametrize("case", [(2, 37, 1032, "bf16", True, 0, 1.0, 0.2), (8, 2, 8192, "bf16", True, 1, 1.0, 0.0),
                                  (4, 400, 8192, "bf16", True, None, 1.0, 0.1), (1, 900, 2048, "fp16", False, 3, 1.0, 0.0)],
                         ids=lambda c: "-".join(str(v) for v in c))
def test_outputs_in_place_of_inputs(car, case):
    k = Case(*case)
    with car.Car(*case[:4]) as c:
        b = k.branch(car)
        want = run_forward(c, k, b, empty)
        xs, res, no = [x.clone() for x in k.xs], k.residual.clone(), torch.empty_like(k.residual)
        c.reduce_branch_residual_rmsnorm(xs, b, res, k.weight, k.eps, res, no, ar_out=xs[-1])
        c.sync()
        assert torch.equal(res, want["residual_out"]) and torch.equal(no, want["norm_out"]) and torch.equal(xs[-1], want["ar"])
        want = run_backward(c, k, b, k.grads(empty))
        for first, second in (("dnorm", "dres"), ("ar", "h"), ("dres", "ar"), ("h", "dnorm")):
            dys, ar, h, dres = [d.clone() for d in k.dys], k.a.clone(), k.h.clone(), k.dres.clone()
            to = {"dnorm": dys[-1], "ar": ar, "h": h, "dres": dres}
            got = {**k.grads(empty), "dx": to[first], "dresidual": to[second]}
            c.reduce_branch_residual_rmsnorm_backward(dys, b, ar, h, k.weight, k.eps, dres, got["dx"], got["dresidual"],
                                                      got["dweight"], got["dnorm_weight"], got["dgate"])
            c.sync()
            assert all(t is None or torch.equal(t, got[name]) for name, t in want.items()), (first, second)


def test_rows_of_zeros_nan_and_infinity(car):
    W, M, N = 2, 9, 512
    k = Case(W, M, N, "bf16", gate_rows=1, p=0.25, eps=1e-4)
    for x in k.xs:
        x[0] = 0                                # nothing behind the norm: h is the residual
    k.xs[0][2, 7] = float("nan")
    k.xs[1][4, 9] = float("inf")
    k.residual[6] = 0
    for x in k.xs:
        x[6] = 0                                # nothing at all: norm_out is 0
    with car.Car(W, M, N, "bf16") as c:
        got = run_forward(c, k, k.branch(car), empty)
        c.sync()
        f = k.factor()
        assert torch.equal(got["residual_out"][0], k.residual[0]) and (got["norm_out"][6] == 0).all()
        for row in (2, 4):  # what is dropped of a row without a norm is 0 all the same
            h = got["residual_out"][row]
            assert torch.equal(h[f[row] == 0], k.residual[row][f[row] == 0])
            assert got["norm_out"][row].isnan().all()
        assert got["residual_out"][2][f[2] != 0].isnan().all()
        rest = [0, 1, 3, 5, 6, 7, 8]
        want = {n: (v[rest], b[rest]) for n, (v, b) in k.forward().items()}
        for name, t in got.items():
            v, b = want[name]
            assert_within(t[rest], v, half("bf16") * v.abs() + 1.01 * b + 2.0**-134, name)
        k.a[3] = 0
        k.h[5] = 0
        got = run_backward(c, k, k.branch(car), k.grads(empty))
        c.sync()
        k.check_backward(got)
        k.h[1, 1] = float("nan")
        got = run_backward(c, k, k.branch(car), k.grads(empty))
        c.sync()
        assert got["dresidual"][1].isnan().all() and got["dweight"].isnan().all()
        keep = [0, 2, 3, 4, 5, 6, 7, 8]
        v, b = k.backward()["dx"]
        assert_within(got["dx"][keep], v[keep], half("bf16") * v[keep].abs() + 1.01 * b[keep] + 2.0**-134, "dx")
        # the gradient of a dropped value is 0 before the norm's own part comes in: a row that is all dropped has none
        k.h[1, 1] = 1.0
        got = run_backward(c, k, k.branch(car, dropout=car.Dropout(1.0, 0)), k.grads(empty))
        c.sync()
        assert (got["dx"] == 0).all() and (got["dgate"] == 0).all() and (got["dnorm_weight"] == 0).all()


def loss(leaves, k, f, dy, dro):
    xs, res, w, w1, gate = leaves
    a = sum(xs)
    y = a * torch.rsqrt((a * a).mean(1, keepdim=True) + k.norm_eps) * w1
    h = k.scale * res + y * gate.repeat_interleave(k.M // gate.shape[0], 0) * f
    return (h * torch.rsqrt((h * h).mean(1, keepdim=True) + k.eps) * w * dy).sum() + (h * dro).sum()


@pytest.mark.parametrize("gate_rows", [1, 3, 0])
def test_matches_autograd_and_differences(car, gate_rows):
    """fp32, eps large enough to matter: autograd of the forward in 64 bits at the stored sum and h, and central
    differences of its loss along random directions.  A step of 1e-4 leaves 1e-8 of the third derivative."""
    W, M, N = 3, 6, 260
    k = Case(W, M, N, "fp32", gate_rows=gate_rows, scale=0.8, p=0.3, eps=0.3)
    f = k.factor()
    xs = [x.double() for x in k.xs]
    k.a = sum(xs).float()
    xs[0] = k.a.double() - sum(xs[1:])      # so that the stored sum is the forward's
    w, w1, gate = k.weight.double(), k.norm_weight.double(), k.gate.double()
    a = k.a.double()
    z = a * torch.rsqrt((a * a).mean(1, keepdim=True) + k.norm_eps) * w1 * k.gates() * f
    k.h = (k.scale * k.residual.double() + z).float()
    res = (k.h.double() - z) / k.scale      # and the stored h
    with car.Car(W, M, N, "fp32") as c:
        got = run_backward(c, k, k.branch(car), k.grads(empty))
        c.sync()
    leaves = [[x.clone().requires_grad_() for x in xs], *(t.clone().requires_grad_() for t in (res, w, w1, gate))]
    dy, dro = rank_sum(k.dys).double(), k.dres.double()
    loss(leaves, k, f, dy, dro).backward()
    bounds = {n: b + half("fp32") * v.abs() for n, (v, b) in k.backward().items()}
    for x in leaves[0]:                      # every rank has the same gradient
        assert_within(got["dx"], x.grad, bounds["dx"], "dx")
    for name, leaf in zip(("dresidual", "dweight", "dnorm_weight", "dgate"), leaves[1:]):
        assert_within(got[name], leaf.grad, bounds[name], name)
    g, e = gen(3), 1e-4
    for _ in range(3):
        v = {n: randn(g, tuple(t.shape), "fp32").double() for n, t in got.items()}
        moved = lambda s: loss([[xs[0] + s * v["dx"], *xs[1:]], res + s * v["dresidual"], w + s * v["dweight"],  # noqa: E731
                                w1 + s * v["dnorm_weight"], gate + s * v["dgate"]], k, f, dy, dro)
        along = sum((got[n].double() * v[n]).sum() for n in v)
        room = sum((bounds[n] * v[n].abs()).sum() for n in v)
        assert abs(along - (moved(e) - moved(-e)) / (2 * e)) <= room + 1e-6 * abs(along)


# the row kernels (whole rows, split rows) and many rows; each shape and type run by no other test
FIRST = [(2, 5, 648, "fp16", True, 5, 1.0, 0.1), (8, 3, 8208, "fp16", True, None, 1.0, 0.0),
         (4, 912, 4112, "fp16", True, 3, 1.0, 0.1), (1, 900, 4120, "fp32", True, 0, 1.0, 0.0)]


def both(c, k, b, fwd, bwd, stream=None, workspace=None):
    c.reduce_branch_residual_rmsnorm(k.xs, b, k.residual, k.weight, k.eps, fwd["residual_out"], fwd["norm_out"],
                                     ar_out=fwd["ar"], stream=stream)
    c.reduce_branch_residual_rmsnorm_backward(k.dys, b, fwd["ar"], fwd["residual_out"], k.weight, k.eps, k.dres, bwd["dx"],
                                              bwd["dresidual"], bwd["dweight"], bwd["dnorm_weight"], bwd["dgate"],
                                              workspace=workspace, stream=stream)


def outputs(k):
    return {n: empty((k.M, k.N), TORCH_DTYPE[k.dtype]) for n in ("residual_out", "norm_out", "ar")}, k.grads(empty)


def same(a, b):
    return all(t is None or torch.equal(t, b[i][n]) for i in range(2) for n, t in a[i].items())


@pytest.mark.parametrize("case", FIRST, ids=lambda c: "-".join(str(v) for v in c))
def test_first_use_in_a_capture(car, case):
    k = Case(*case)
    captured, eager = outputs(k), outputs(k)
    with car.Car(*case[:4]) as c, car.Car(*case[:4]) as other:
        b = k.branch(car)
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            both(c, k, b, *captured)
        graph.replay()
        c.sync()
        both(other, k, b, *eager)
        other.sync()
        k.check_forward(captured[0])
        assert same(captured, eager)
        del graph


@pytest.mark.parametrize("case", FIRST, ids=lambda c: "-".join(str(v) for v in c))
def test_first_use_in_two_threads(car, case):
    k = Case(*case)
    outs, want, failed = [outputs(k) for _ in range(2)], outputs(k), []
    with car.Car(*case[:4]) as c, car.Car(*case[:4]) as other:
        b = k.branch(car)
        both(other, k, b, *want)
        ws = [torch.empty(other.branch_workspace_bytes(b), dtype=torch.uint8, device=DEV) for _ in range(2)]
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        gate = threading.Barrier(2)

        def go(i):
            try:
                gate.wait(10)
                both(c, k, b, *outs[i], stream=streams[i], workspace=ws[i])
            except Exception as e:  # noqa: BLE001
                failed.append(e)

        ts = [threading.Thread(target=go, args=(i,)) for i in range(2)]
        for t in ts:
            t.start()
        for t in ts:
            t.join()
        torch.cuda.synchronize()
        c.sync()
        assert not failed and same(want, outs[0]) and same(want, outs[1])


def test_captured_with_its_own_workspace_and_new_masks(car):
    """Two graphs of one handle, each with a workspace from its own pool, replayed in turn with new inputs and offsets."""
    W, M, N = 4, 300, 2056
    k = Case(W, M, N, "bf16", gate_rows=5, p=0.2)
    step = torch.zeros(1, dtype=torch.int64, device=DEV)
    outs, graphs = [outputs(k) for _ in range(2)], []
    with car.Car(W, M, N, "bf16") as c:
        b = k.branch(car, dropout=car.Dropout(k.p, k.seed, k.offset, offset_dev=step))
        torch.cuda.synchronize()
        for o in outs:
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=torch.cuda.Stream()):
                both(c, k, b, *o)
        for seed in (13, 14):
            new = Case(W, M, N, "bf16", gate_rows=5, p=0.2, seed=seed)
            for a, x in zip([*k.xs, *k.dys, k.residual, k.dres, k.weight, k.norm_weight, k.gate],
                            [*new.xs, *new.dys, new.residual, new.dres, new.weight, new.norm_weight, new.gate]):
                a.copy_(x)
            for graph, o in zip(graphs, outs):
                step.add_(1)
                k._factor = factor(M, N, k.p, k.seed, (k.offset + int(step)) % 2**64)
                graph.replay()
                c.sync()
                k.check_forward(o[0])
                k.a, k.h = o[0]["ar"], o[0]["residual_out"]
                k.check_backward(o[1])
        del graphs


def test_two_streams_at_once_with_two_workspaces(car):
    W, M, N = 2, 500, 4096
    ks = [Case(W, M, N, "bf16", gate_rows=1, p=0.1, seed=31 + i) for i in range(2)]
    outs, streams = [outputs(k) for k in ks], [torch.cuda.Stream() for _ in range(2)]
    with car.Car(W, M, N, "bf16") as c:
        bs = [k.branch(car) for k in ks]
        ws = [torch.empty(c.branch_workspace_bytes(b), dtype=torch.uint8, device=DEV) for b in bs]
        torch.cuda.synchronize()
        for _ in range(5):
            for k, b, o, s, w in zip(ks, bs, outs, streams, ws):
                both(c, k, b, *o, stream=s, workspace=w)
        torch.cuda.synchronize()
        for k, o in zip(ks, outs):
            k.check_forward(o[0])
            k.a, k.h = o[0]["ar"], o[0]["residual_out"]
            k.check_backward(o[1])
        with pytest.raises(ValueError):  # no workspace to be had for a stream that is not the current one
            both(c, ks[0], bs[0], *outs[0], stream=streams[0])


def test_the_same_rank_twice_and_distinct_handles(car):
    """One buffer given as two ranks is added twice; handles of other shapes in between change nothing."""
    W, M, N = 4, 200, 8192
    k = Case(W, M, N, "bf16")
    k.xs = [k.xs[0], k.xs[1], k.xs[0], k.xs[1]]
    k.dys = [k.dys[0]] * W
    o = outputs(k)
    with car.Car(W, M, N, "bf16") as c, car.Car(2, 900, 1024, "bf16") as d:
        other = Case(2, 900, 1024, "bf16", p=0.1)
        for _ in range(2):
            both(c, k, k.branch(car), *o)
            p = outputs(other)
            both(d, other, other.branch(car), *p)
        c.sync()
        d.sync()
        k.check_forward(o[0])
        other.check_forward(p[0])
        k.a, k.h = o[0]["ar"], o[0]["residual_out"]
        k.check_backward(o[1])


@pytest.mark.parametrize("which", ["forward", "backward"])
def test_wait_that_runs_out_is_reported(car, which):
    """One CTA of a split row is late by more than the wait's limit: car_sync reports it, the row has NaN, the other rows
    are as ever, and so is the next call."""
    W, M, N = 8, 2, 8192
    k = Case(W, M, N, "bf16", gate_rows=0)
    with car.Car(W, M, N, "bf16") as c:
        b = k.branch(car)
        go = (lambda: run_forward(c, k, b, empty)) if which == "forward" else (lambda: run_backward(c, k, b, k.grads(empty)))
        want = go()
        c.sync()
        car.check(car.car_test_delay_partial(c.h, 20000, 2, 1, 3000000))
        got = go()
        with pytest.raises(car.CarError) as e:
            c.sync()
        assert e.value.status == car.CAR_ERR_TIMEOUT
        row = "norm_out" if which == "forward" else "dx"
        assert got[row][1].isnan().any() and torch.equal(got[row][0], want[row][0])
        car.check(car.car_test_delay_partial(c.h, 0, -1, 0, 0))
        got = go()
        c.sync()
        assert all(t is None or torch.equal(t, got[n]) for n, t in want.items())


@pytest.mark.parametrize("which", ["forward", "backward"])
@pytest.mark.parametrize("W,M,N,cta", [(2, 160, 16384, 1), (1, 170, 32768, 3)])
def test_wait_of_a_split_row_in_the_pipeline(car, which, W, M, N, cta):
    """The same where the pipeline's CTAs share a row."""
    k = Case(W, M, N, "bf16")
    with car.Car(W, M, N, "bf16") as c:
        b = k.branch(car)
        go = (lambda: run_forward(c, k, b, empty)) if which == "forward" else (lambda: run_backward(c, k, b, k.grads(empty)))
        want = go()
        c.sync()
        car.check(car.car_test_delay_partial(c.h, 20000, cta, 7, 3000000))
        got = go()
        with pytest.raises(car.CarError) as e:
            c.sync()
        assert e.value.status == car.CAR_ERR_TIMEOUT
        row, rest = "norm_out" if which == "forward" else "dx", [m for m in range(M) if m != 7]
        assert got[row][7].isnan().any() and torch.equal(got[row][rest], want[row][rest])
        car.check(car.car_test_delay_partial(c.h, 0, -1, 0, 0))
        got = go()
        c.sync()
        assert all(t is None or torch.equal(t, got[n]) for n, t in want.items())


# both sides of the borders between the row kernels and the pipelines (152 SMs), and between whole and split rows
BORDERS = [(1, 455, 1024, "bf16"), (1, 456, 1024, "bf16"), (4, 455, 2048, "fp16"), (4, 456, 2048, "fp16"), (8, 227, 8192, "bf16"),
           (8, 228, 8192, "bf16"), (16, 303, 8192, "fp16"), (16, 304, 8192, "fp16"), (2, 151, 8200, "bf16"), (2, 152, 8200, "bf16"),
           (2, 153, 8192, "bf16"), (1, 303, 1024, "bf16"), (1, 304, 1024, "bf16"), (3, 304, 6152, "bf16"), (1, 152, 12288, "bf16"),
           (1, 152, 12296, "bf16"), (1, 160, 16384, "bf16"), (1, 160, 16392, "bf16"), (1, 153, 8196, "fp32"), (2, 160, 16384, "fp32")]


@pytest.mark.parametrize("W,M,N,dtype", BORDERS)
def test_borders_between_kernels(car, W, M, N, dtype):
    k = Case(W, M, N, dtype, gate_rows=M % 2, p=0.1 if M % 3 else 0.0)
    with car.Car(W, M, N, dtype) as c:
        b = k.branch(car)
        got, grads = run_forward(c, k, b, empty), run_backward(c, k, b, k.grads(empty))
        c.sync()
    k.check_forward(got)
    k.check_backward(grads)


@pytest.mark.parametrize("case", [(2, 37, 1032, "bf16", True, 37, 1.0, 0.2), (4, 400, 4096, "fp32", True, 4, 1.0, 0.0),
                                  (1, 900, 2048, "fp16", False, 3, 1.0, 0.0), (1, 310, 2056, "bf16", True, 0, 1.0, 0.1),
                                  (2, 160, 12296, "bf16", True, 1, 1.0, 0.0)], ids=lambda c: "-".join(str(v) for v in c))
def test_every_gradient_may_be_left_out(car, case):
    """The others keep their bits, and nothing is written in its place."""
    k = Case(*case)
    with car.Car(*case[:4]) as c:
        b = k.branch(car)
        want = run_backward(c, k, b, k.grads(empty))
        for name in ("dresidual", "dweight", "dnorm_weight", "dgate"):
            for alone in (False, True):
                got = k.grads(empty)
                for other in ("dresidual", "dweight", "dnorm_weight", "dgate"):
                    if (other == name) != alone:
                        got[other] = None
                run_backward(c, k, b, got)
                c.sync()
                assert all(t is None or torch.equal(t, want[n]) for n, t in got.items()), (name, alone)


def test_rows_past_32_bits_of_elements(car):
    """4.3 billion elements: the last rows, forward and backward, against the formulas."""
    W, M, N = 1, 2**19 + 5, 8192
    last = slice(M - 4, M)
    g = gen(17)
    x = torch.ones(M, N, device=DEV, dtype=torch.bfloat16)
    res, dy = torch.ones_like(x), torch.ones_like(x)
    small = Case(W, 4, N, "bf16", skip=False)
    x[last], res[last], dy[last] = small.xs[0], small.residual, small.dys[0]
    weight, norm_weight = small.weight, small.norm_weight
    ro, no, ar = (torch.empty_like(x) for _ in range(3))
    drop = car.Dropout(0.25, 5, 6)
    with car.Car(W, M, N, "bf16") as c:
        b = car.Branch(norm_weight, small.norm_eps, dropout=drop)
        c.reduce_branch_residual_rmsnorm([x], b, res, weight, small.eps, ro, no, ar_out=ar)
        c.reduce_branch_residual_rmsnorm_backward([dy], b, ar, ro, weight, small.eps, None, x, res)
        c.sync()
    import numpy as np

    from branch_checks import philox

    at = np.arange((M - 4) * N // 8, M * N // 8, dtype=np.uint64)
    words = np.stack([at % 2**32, at >> np.uint64(32), np.full_like(at, 6), np.zeros_like(at)], 1)
    w = philox(words, (5, 0))
    kept = np.stack([w & 0xFFFF, w >> 16], 2).reshape(4, N) >= 16384
    small._factor, small.p = torch.from_numpy(kept * (65536 / 49152)).to(DEV), 0.25
    small.check_forward({"ar": ar[last], "residual_out": ro[last], "norm_out": no[last]})
    small.a, small.h = ar[last], ro[last]
    small.check_backward({"dx": x[last], "dresidual": res[last]})


def test_more_rows_than_a_pipeline_counts(car):
    """1025 times the same 2^20 rows of one vector: the same results 1025 times, the first ones those of the formulas."""
    P, N, W = 2**20, 8, 1
    M = 1025 * P
    small = Case(W, 4, N, "bf16", skip=False)

    def repeated(first, seed):
        rows = randn(gen(seed), (P, N), "bf16")
        rows[:4] = first
        return rows.expand(1025, P, N).contiguous().view(M, N)

    def first_rows(t):
        parts = t.view(1025, P, N)
        assert all(torch.equal(parts[0], parts[i]) for i in range(1, 1025))
        return parts[0][:4]

    with car.Car(W, M, N, "bf16") as c:
        b = car.Branch(small.norm_weight, small.norm_eps)
        x, res = repeated(small.xs[0], 3), repeated(small.residual, 4)
        no = torch.empty_like(x)
        c.reduce_branch_residual_rmsnorm([x], b, res, small.weight, small.eps, res, no, ar_out=x)
        c.sync()
        a, h = first_rows(x).clone(), first_rows(res).clone()
        small.check_forward({"ar": a, "residual_out": h, "norm_out": first_rows(no)})
        dy = repeated(small.dys[0], 5)
        c.reduce_branch_residual_rmsnorm_backward([dy], b, x, res, small.weight, small.eps, None, dy, no)
        c.sync()
        small.a, small.h = a, h
        small.check_backward({"dx": first_rows(dy), "dresidual": first_rows(no)})


def test_refusals(car):
    W, M, N = 2, 400, 64
    k = Case(W, M, N, "bf16", gate_rows=4)
    o, gr = outputs(k)
    with car.Car(W, M, N, "bf16") as c:
        b = k.branch(car)
        ws = torch.empty(c.branch_workspace_bytes(b), dtype=torch.uint8, device=DEV)
        P = lambda t: t.data_ptr()  # noqa: E731
        br = lambda **ch: car.car_branch(**{**dict(norm_weight=P(k.norm_weight), norm_eps=1e-6, gate=P(k.gate),  # noqa: E731
                                                   gate_rows=4, residual_scale=1.0), **ch})
        fwd = dict(h=c.h, inputs=[P(x) for x in k.xs], branch=br(), residual=P(k.residual), weight=P(k.weight), eps=1e-6,
                   residual_out=P(o["residual_out"]), norm_out=P(o["norm_out"]), ar_out=P(o["ar"]))
        out = lambda **ch: car.car_branch_grads(**{**{n: P(t) for n, t in gr.items()}, **ch})  # noqa: E731
        bwd = dict(h=c.h, dnorm=[P(d) for d in k.dys], branch=br(), ar=P(k.a), residual_out=P(k.h), weight=P(k.weight),
                   eps=1e-6, dresidual_out=P(k.dres), out=out(), workspace=P(ws))
        F = lambda **ch: car.car_reduce_branch_residual_rmsnorm(**{**fwd, **ch})  # noqa: E731
        B = lambda **ch: car.car_reduce_branch_residual_rmsnorm_backward(**{**bwd, **ch})  # noqa: E731
        nan, inf = float("nan"), float("inf")
        drop = car.car_dropout(2.0, 0, 0, None)
        import ctypes

        bad_branches = [br(gate_rows=3), br(gate_rows=-1), br(gate_rows=401), br(residual_scale=nan), br(residual_scale=inf),
                        br(norm_eps=-1.0), br(norm_eps=nan), br(dropout=ctypes.pointer(drop)), None]
        for call in (F, B):
            for bad in bad_branches:
                assert call(branch=bad) == car.CAR_ERR_ARG
            for eps in (-1.0, nan, inf):
                assert call(eps=eps) == car.CAR_ERR_ARG
            assert call(branch=br(gate=P(k.gate) + 2)) == car.CAR_ERR_ALIGN
            assert call(branch=br(norm_weight=P(k.norm_weight) + 2)) == car.CAR_ERR_ALIGN
            assert call(weight=None) == car.CAR_ERR_ARG and call(weight=P(k.weight) + 4) == car.CAR_ERR_ALIGN
        assert F(inputs=None) == car.CAR_ERR_ARG and F(residual=None) == car.CAR_ERR_ARG and F(norm_out=None) == car.CAR_ERR_ARG
        assert F(residual_out=None) == car.CAR_ERR_ARG and F(ar_out=P(o["ar"]) + 2) == car.CAR_ERR_ALIGN
        # overlaps: two outputs, an output over an input that it may not replace or only in part
        D = M * N * 2
        for ch in (dict(norm_out=P(o["residual_out"])), dict(ar_out=P(o["norm_out"])), dict(norm_out=P(k.xs[0])),
                   dict(norm_out=P(k.residual)), dict(residual_out=P(k.xs[1])), dict(residual_out=P(k.residual) + 16),
                   dict(ar_out=P(k.xs[0]) + D - 16), dict(ar_out=P(k.residual)), dict(norm_out=P(k.gate)),
                   dict(residual_out=P(k.weight))):
            assert F(**ch) == car.CAR_ERR_ARG, ch
        assert B(dnorm=None) == car.CAR_ERR_ARG and B(residual_out=None) == car.CAR_ERR_ARG and B(out=None) == car.CAR_ERR_ARG
        assert B(out=out(dx=None)) == car.CAR_ERR_ARG and B(workspace=None) == car.CAR_ERR_ARG and B(ar=None) == car.CAR_ERR_ARG
        assert B(branch=br(norm_weight=None)) == car.CAR_ERR_ARG     # a dnorm_weight without a norm
        assert B(branch=br(gate=None)) == car.CAR_ERR_ARG            # a dgate without a gate
        for n in ("dx", "dresidual", "dweight", "dnorm_weight", "dgate"):
            assert B(out=out(**{n: P(gr[n]) + 4})) == car.CAR_ERR_ALIGN
        assert B(workspace=P(ws) + 8) == car.CAR_ERR_ALIGN and B(ar=P(k.a) + 2) == car.CAR_ERR_ALIGN
        assert B(dresidual_out=P(k.dres) + 2) == car.CAR_ERR_ALIGN
        for ch in (dict(dx=P(gr["dresidual"])), dict(dx=P(k.a) + 16), dict(dresidual=P(k.gate)), dict(dweight=P(k.h)),
                   dict(dgate=P(ws)), dict(dnorm_weight=P(gr["dweight"])), dict(dresidual=P(k.weight))):
            assert B(out=out(**ch)) == car.CAR_ERR_ARG, ch
        assert B(workspace=P(k.h)) == car.CAR_ERR_ARG
        # what is not asked for needs nothing
        none = dict(dweight=None, dnorm_weight=None, dgate=None, dresidual=None)
        assert B(out=out(**none), workspace=None) == car.CAR_OK
        assert B(out=out(**none), workspace=None, branch=br(norm_weight=None), ar=None) == car.CAR_OK
        assert F(ar_out=None, branch=br(norm_weight=None, norm_eps=nan)) == car.CAR_OK   # norm_eps is not read
        assert car.car_branch_workspace_bytes(c.h, br(gate_rows=3)) == 0
        for kw in (dict(workspace=ws[:-1]),):
            with pytest.raises(ValueError):
                run_backward(c, k, b, gr, **kw)
        with pytest.raises(ValueError):
            c.reduce_branch_residual_rmsnorm(k.xs, car.Branch(gate=k.gate[:3], gate_rows=4), k.residual, k.weight, 1e-6,
                                             o["residual_out"], o["norm_out"])
        with pytest.raises(ValueError):
            c.reduce_branch_residual_rmsnorm(k.xs, car.Branch(norm_weight=k.norm_weight[:-1]), k.residual, k.weight, 1e-6,
                                             o["residual_out"], o["norm_out"])
        c.sync()
    with car.Car(1, 1, 65536, "bf16") as c:   # a row of 128 KB
        t = torch.empty(1, 65536, dtype=torch.bfloat16, device=DEV)
        for call in (lambda: c.reduce_branch_residual_rmsnorm([t], car.Branch(), t, t, 1e-6, t, t.clone()),
                     lambda: c.reduce_branch_residual_rmsnorm_backward([t], car.Branch(), None, t, t, 1e-6, None, t)):
            with pytest.raises(car.CarError) as e:
                call()
            assert e.value.status == car.CAR_ERR_SIZE
        assert c.branch_workspace_bytes() == 0
        drop = torch.empty_like(t)
        c.reduce_dropout([t.fill_(1.0)], car.Dropout(0.5, 1), drop)   # has no such limit
        c.sync()
        assert set(drop.unique().tolist()) == {0.0, 2.0}
