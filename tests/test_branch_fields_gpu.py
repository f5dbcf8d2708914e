"""A branch whose tensors, gate rows and dropout change between calls: each call against the formulas in 64 bits (tolerances:
see branch_checks), as a call with a branch made anew."""
import pytest
import torch

from branch_checks import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def car():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import rank_sum_reduce_gb300 as car

    return car


def run(c, k, b):
    fwd = {n: torch.empty_like(k.residual) for n in ("residual_out", "norm_out", "ar")}
    c.reduce_branch_residual_rmsnorm(k.xs, b, k.residual, k.weight, k.eps, fwd["residual_out"], fwd["norm_out"], ar_out=fwd["ar"])
    bwd = k.grads(lambda shape, dtype: torch.empty(shape, dtype=dtype, device="cuda"))
    c.reduce_branch_residual_rmsnorm_backward(k.dys, b, k.a, k.h, k.weight, k.eps, k.dres, bwd["dx"], bwd["dresidual"],
                                              bwd["dweight"], bwd["dnorm_weight"], bwd["dgate"])
    c.sync()
    k.check_forward(fwd)
    k.check_backward(bwd)


def test_fields_set_between_calls(car):
    W, M, N = 2, 480, 1032
    k = Case(W, M, N, "bf16", gate_rows=1, p=0.1)
    with car.Car(W, M, N, "bf16") as c:
        b = k.branch(car)
        run(c, k, b)
        for gate_rows, p in ((480, 0.0), (0, 0.3), (6, 0.3)):
            k = Case(W, M, N, "bf16", gate_rows=gate_rows, p=p, scale=0.5, seed=gate_rows)
            b.norm_weight, b.gate, b.gate_rows, b.residual_scale = k.norm_weight, k.gate, gate_rows, 0.5
            b.dropout = car.Dropout(p, k.seed, k.offset) if p else None
            run(c, k, b)


def test_parameters_whose_data_is_exchanged(car):
    W, M, N = 4, 9, 2056
    k = Case(W, M, N, "fp16", gate_rows=3)
    w, g = (torch.nn.Parameter(t.clone()) for t in (k.norm_weight, k.gate))
    with car.Car(W, M, N, "fp16") as c:
        b = k.branch(car, norm_weight=w, gate=g)
        run(c, k, b)
        k = Case(W, M, N, "fp16", gate_rows=3, seed=5)
        w.data, g.data = k.norm_weight.clone(), k.gate.clone()
        run(c, k, b)
