"""The branch backward's sums over very many rows, which take several launches, against the formulas in 64 bits.

Tolerances: branch_checks allows 128 roundings of 2^-24 for a sum; here a thread adds 512 rows one after the other, 16 teams and
304 partials in a tree of 48 more, and then every launch's sum is added to the ones before: 576 and the number of launches.  The
bounds of branch_checks are multiplied by that over 128 (their other terms are not larger for it).  A launch has at least 128 rows
a thread, so there are at most rows / (128 * threads that share a column) of them; a team whose tile has no row for it counts as
none (tiles end with a gate row)."""
import pytest
import torch

from branch_checks import Case
from operator_checks import DEV, assert_within

pytestmark = pytest.mark.gpu

SUMS = ("dweight", "dnorm_weight", "dgate")


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


def roundings(M, adders):
    return 576 + M / (128 * adders)


def backward(c, k, b, got, ar=None, dys=None, h=None, dres=None, **kw):
    c.reduce_branch_residual_rmsnorm_backward(dys or k.dys, b, k.a if ar is None else ar, k.h if h is None else h, k.weight, k.eps,
                                              dres if dres is not None else k.dres, got["dx"], got["dresidual"], got["dweight"],
                                              got["dnorm_weight"], got["dgate"], **kw)


# 16 teams of a warp, or as many CTAs as there are clusters of two (76): a launch takes 1.2 million rows, or 39,000
CASES = [(1, 2737021, 8, "bf16", True, None, 1.0, 0.1), (1, 2737020, 8, "bf16", True, 1, 1.0, 0.0), (2, 2737020, 8, "fp16", True, 3, 1.0, 0.2),
         (1, 2737020, 8, "bf16", False, 20, 1.0, 0.0), (1, 2737020, 8, "fp16", True, 1368510, 1.0, 0.1), (1, 2737020, 8, "bf16", True, 0, 0.5, 0.1),
         (1, 3000001, 4, "fp32", True, None, 1.0, 0.3), (1, 2600000, 4, "fp32", False, 2, 1.0, 0.3), (2, 83333, 4100, "fp32", True, 1, 1.0, 0.1),
         (1, 83334, 4100, "fp32", True, 6, 1.0, 0.0)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_several_launches_match_the_formula(car, case):
    W, M, N = case[:3]
    k = Case(*case)
    with car.Car(*case[:4]) as c:
        b, got = k.branch(car), k.grads(empty)
        backward(c, k, b, got)
        c.sync()
        wide = roundings(M, min(16, M // (k.gate_rows or 1)) * 152 if N < 64 else 76) / 128
        for name, (v, bound) in k.backward().items():
            t = got[name]
            if name in SUMS and t.dtype == torch.float32:
                assert_within(t, v, wide * bound + 2.0**-24 * v.abs(), name)
            elif t is not None:
                k.check_backward({name: t})
        again = k.grads(empty)
        backward(c, k, b, again)                  # the same bits
        for name in ("dresidual",) + SUMS:        # and whatever else is asked for
            alone = {**dict.fromkeys(got), "dx": empty((M, N), k.h.dtype), name: k.grads(empty)[name]}
            backward(c, k, b, alone)
            c.sync()
            assert torch.equal(alone["dx"], got["dx"]) and (got[name] is None or torch.equal(alone[name], got[name]))
        assert all(t is None or torch.equal(t, again[name]) for name, t in got.items())


def alike(car, M, gate_rows, dtype="bf16"):
    """Every row the same: each addition to a sum rounds the same way as the one before, so the error of one sum over all
    rows would grow with their number.  The exact sums are multiples of one row's."""
    W, N = 1, 8
    k = Case(W, 1, N, dtype, gate_rows=1, skip=False, seed=7)
    rows = lambda t: t.expand(M, N).contiguous()  # noqa: E731
    k.h.abs_().add_(0.5)
    k.a.abs_().add_(0.5)
    k.dys[0].abs_().add_(0.5)
    got = {"dx": rows(k.dys[0]), "dresidual": None, "dweight": empty((N,), torch.float32), "dnorm_weight": empty((N,), torch.float32)}
    got["dgate"] = empty((gate_rows, N), torch.float32)
    gate = k.gate.expand(gate_rows, N).contiguous()
    with car.Car(W, M, N, dtype) as c:
        b = k.branch(car, gate=gate, gate_rows=gate_rows)
        backward(c, k, b, got, ar=rows(k.a), dys=[got["dx"]], h=rows(k.h))
        c.sync()
    assert torch.equal(got["dx"], got["dx"][:1].expand(M, N))
    wide = roundings(M, min(16, M // gate_rows) * 152) / 128
    for name in SUMS:
        v, bound = k.backward()[name]
        times = M // gate_rows if name == "dgate" else M
        assert_within(got[name], (times * v).expand(got[name].shape), (wide * times * bound).expand(got[name].shape), name)


@pytest.mark.parametrize("gate_rows", [1, 5, 30, 6000000, 15000000])
def test_rows_that_are_all_alike(car, gate_rows):
    alike(car, 30000000, gate_rows)


def test_more_than_2_to_the_30_rows(car):
    alike(car, 1025 * 2**20, 1025)


@pytest.mark.parametrize("case", [(1, 2737020, 8, "bf16", True, 1, 1.0, 0.1), (1, 2737020, 8, "bf16", True, 30, 1.0, 0.1)],
                         ids=lambda c: "-".join(str(v) for v in c))
def test_captured_and_in_place(car, case):
    k = Case(*case)
    with car.Car(*case[:4]) as c:
        b, want, got = k.branch(car), k.grads(empty), k.grads(empty)
        backward(c, k, b, want)
        c.sync()
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            backward(c, k, b, got)
        for _ in range(2):
            graph.replay()
            c.sync()
            assert all(t is None or torch.equal(t, got[name]) for name, t in want.items())
        del graph
        dys, h = [d.clone() for d in k.dys], k.h.clone()
        got["dx"], got["dresidual"] = dys[0], h
        backward(c, k, b, got, dys=dys, h=h)
        c.sync()
        assert all(t is None or torch.equal(t, got[name]) for name, t in want.items())
