"""Waits of a split row that run out (a CTA is late by more than the limit, both bounded): what the outputs hold then.
Dropped elements stay finite where the statistic is multiplied in before the dropout, and in the pipeline the row that the
CTA had before the late one loses its norm_out with it."""
import pytest
import torch

from branch_checks import Case
from operator_checks import DEV

pytestmark = pytest.mark.gpu

LIMIT, LATE = 20000, 3000000   # ns


@pytest.fixture(scope="module")
def car():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import rank_sum_reduce_gb300 as car

    return car


def forward(c, k, b):
    got = {n: torch.empty_like(k.residual) for n in ("residual_out", "norm_out", "ar")}
    c.reduce_branch_residual_rmsnorm(k.xs, b, k.residual, k.weight, k.eps, got["residual_out"], got["norm_out"], ar_out=got["ar"])
    return got


def backward(c, k, b):
    got = k.grads(lambda shape, dtype: torch.empty(shape, dtype=dtype, device=DEV))
    c.reduce_branch_residual_rmsnorm_backward(k.dys, b, k.a if k.needs_sum else None, k.h, k.weight, k.eps, k.dres, got["dx"],
                                              got["dresidual"], got["dweight"], got["dnorm_weight"], got["dgate"])
    return got


def late(car, k, call, cta, row):
    """What the call gives, and what it gives when this CTA is late for this row; the call after that is as the first."""
    with car.Car(k.W, k.M, k.N, k.dtype) as c:
        b = k.branch(car)
        want = call(c, k, b)
        c.sync()
        car.check(car.car_test_delay_partial(c.h, LIMIT, cta, row, LATE))
        got = call(c, k, b)
        with pytest.raises(car.CarError) as e:
            c.sync()
        assert e.value.status == car.CAR_ERR_TIMEOUT
        car.check(car.car_test_delay_partial(c.h, 0, -1, 0, 0))
        again = call(c, k, b)
        c.sync()
        assert all(t is None or torch.equal(t, again[n]) for n, t in want.items())
    return want, got


def rows_that_differ(a, b):
    bits = {2: torch.int16, 4: torch.int32}[a.element_size()]
    return (a.view(bits) != b.view(bits)).any(1).nonzero().flatten().tolist()


@pytest.mark.parametrize("W,M,N,cta", [(2, 160, 16384, 1), (1, 170, 32768, 3), (2, 400, 13000, 0)])
def test_a_row_behind_the_first_of_its_cluster(car, W, M, N, cta):
    """There are at most 76 clusters of two, or 38 of four: the last row is never its cluster's first.  The row before it
    in its cluster loses its norm_out, whose sum travels with the late exchange; nothing else of it."""
    k = Case(W, M, N, "bf16")
    want, got = late(car, k, forward, cta, M - 1)
    assert rows_that_differ(want["ar"], got["ar"]) == []
    assert rows_that_differ(want["residual_out"], got["residual_out"]) == [M - 1]
    rows = rows_that_differ(want["norm_out"], got["norm_out"])
    assert len(rows) == 2 and rows[1] == M - 1 and rows[0] >= M - 1 - 76
    for row in rows:
        assert got["norm_out"][row].isnan().any()
        same = got["norm_out"][row] == want["norm_out"][row]
        assert (same | got["norm_out"][row].isnan()).all()
    assert got["norm_out"][M - 1].isnan().all()      # a NaN of h is in its row's second sum
    assert not got["norm_out"][rows[0]].isnan().all()  # the late CTA had its peers' parts


@pytest.mark.parametrize("W,M,N,cta,row", [(8, 2, 8192, 2, 1), (2, 160, 16384, 1, 7), (1, 170, 32768, 3, 100)])
def test_dropped_elements_of_the_forward_stay_finite(car, W, M, N, cta, row):
    k = Case(W, M, N, "bf16", gate_rows=0, p=0.3, scale=0.5)
    want, got = late(car, k, forward, cta, row)
    dropped, h = k.factor()[row] == 0, got["residual_out"][row]
    assert rows_that_differ(want["residual_out"], got["residual_out"]) == [row]
    assert torch.equal(h[dropped], want["residual_out"][row][dropped])
    assert torch.equal(h[dropped], (0.5 * k.residual[row].float()).bfloat16()[dropped])
    assert h[~dropped].isnan().any() and (h.isnan() | (h == want["residual_out"][row])).all()
    assert got["norm_out"][row].isnan().all()


@pytest.mark.parametrize("W,M,N,cta,row", [(8, 2, 8192, 2, 1), (2, 160, 16384, 1, 7), (1, 170, 32768, 3, 169)])
@pytest.mark.parametrize("norm", [False, True])
def test_dropped_elements_of_the_backward(car, W, M, N, cta, row, norm):
    """Without a norm they are 0 as ever; with one the second sum's NaN reaches the whole row."""
    k = Case(W, M, N, "bf16", norm=norm, p=0.3)
    want, got = late(car, k, backward, cta, row)
    dropped, dx, dr = k.factor()[row] == 0, got["dx"][row], got["dresidual"][row]
    assert rows_that_differ(want["dx"], got["dx"]) == [row] and rows_that_differ(want["dresidual"], got["dresidual"]) == [row]
    lost = dr.isnan()
    assert lost.any() and not lost.all() and (lost | (dr == want["dresidual"][row])).all()
    assert torch.equal(got["dweight"].isnan(), lost)
    if norm:
        assert dx.isnan().all()
    else:
        assert torch.equal(dx.isnan(), lost & ~dropped) and (dx[dropped] == 0).all()
        assert (dx.isnan() | (dx == want["dx"][row])).all()
