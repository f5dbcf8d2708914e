"""Host-side checks of the types that the calls with an 8-bit output or a weight gradient take.  No test here launches
a kernel."""
import pytest


@pytest.fixture(scope="module")
def car():
    import __graft_entry__

    __graft_entry__.build()
    import rank_sum_reduce_gb300 as car

    return car


@pytest.mark.parametrize("kind,bad", [("mx32", "float32"), ("mx32", "int64"), ("row", "float64"), ("row", "uint8"),
                                      ("group128", "bfloat16"), ("static", "float16")])
def test_scales_of_another_type_are_refused(car, kind, bad):
    """Before any pointer is taken: large enough tensors whose values would be read or written as something else."""
    import torch

    c = object.__new__(car.Car)   # the check needs no handle
    c.h = None
    t, q = torch.empty(4, 64, dtype=torch.bfloat16), torch.empty(4, 64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="scales: torch." + bad):
        c.reduce_residual_rmsnorm_quant([t], t, t[0], 1e-6, kind, t, q, torch.empty(64, dtype=getattr(torch, bad)))


def test_codes_and_weight_gradients_of_another_type_are_refused(car):
    import torch

    c = object.__new__(car.Car)
    c.h = None
    t = torch.empty(4, 64, dtype=torch.bfloat16)
    for bad in (torch.bfloat16, torch.float8_e5m2, torch.float32):
        with pytest.raises(ValueError, match="q_out"):
            c.reduce_residual_rmsnorm_quant([t], t, t[0], 1e-6, "row", t, t.to(bad), torch.empty(4))
    for bad in (torch.float64, torch.bfloat16, torch.int64):
        with pytest.raises(ValueError, match="dweight"):
            c.reduce_residual_rmsnorm_backward([t], t, t[0], 1e-6, None, t, torch.empty(64, dtype=bad))
