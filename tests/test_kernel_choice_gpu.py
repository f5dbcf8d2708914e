"""Rows at the borders where the 8-bit output and the backward go from one kernel to another (rank counts and lengths
that the other tests of these operators take only on one side)."""
import pytest
import torch

import test_norm_backward_gpu as backward
import test_norm_quant_gpu as quant
from operator_checks import DEV, TORCH_DTYPE, Guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def car():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import rank_sum_reduce_gb300 as car

    return car


# eight vectors per thread (rows of more than 56 KB) with eight ranks, at and below one row per SM
@pytest.mark.parametrize("W,M,N,dtype", [(8, 151, 14600, "fp32"), (8, 153, 14600, "fp32"), (8, 311, 16384, "fp32"),
                                         (8, 157, 32768, "bf16"), (8, 153, 29000, "fp16"), (4, 151, 29000, "bf16")])
@pytest.mark.parametrize("kind", ["row", "mx32", "group128"])
def test_quant(car, W, M, N, dtype, kind):
    xs, res, w = quant.make(W, M, N, dtype, seed=W + M + N)
    h, y = quant.normalised(xs, res, w, 1e-6)
    out = Guarded()
    ro, q = out.empty((M, N), TORCH_DTYPE[dtype]), out.empty((M, N), torch.float8_e4m3fn)
    with car.Car(W, M, N, dtype) as c:
        s = out.empty(c.quant_scales_shape(kind), torch.uint8 if kind == "mx32" else torch.float32)
        c.reduce_residual_rmsnorm_quant(xs, res, w, 1e-6, kind, ro, q, s)
        c.sync()
    quant.check_codes(q, y / quant.check_scales(kind, s, y), "q")
    assert torch.equal(ro, h.to(ro.dtype))
    out.check()


# seven vectors per thread with eight ranks, eight with one and sixteen, four 16-bit ones by ranks and warps
@pytest.mark.parametrize("W,M,N,dtype", [
    (8, 151, 12900, "fp32"), (8, 153, 12900, "fp32"), (8, 307, 13320, "fp32"), (1, 1215, 14600, "fp32"), (1, 1217, 14600, "fp32"),
    (16, 1217, 14600, "fp32"), (2, 1217, 14600, "fp32"), (8, 151, 12400, "bf16"), (8, 153, 12400, "bf16"), (16, 161, 14336, "fp16"),
    (16, 161, 14344, "fp16"), (4, 913, 14000, "bf16"), (2, 913, 14000, "bf16")])
def test_backward(car, W, M, N, dtype):
    dys, h, w, dres = backward.make(W, M, N, dtype, seed=W + M + N)
    out = Guarded()
    dx, dw = out.empty((M, N), TORCH_DTYPE[dtype]), out.empty((N,), torch.float32)
    with car.Car(W, M, N, dtype) as c:
        ws = torch.empty(c.backward_workspace_bytes, dtype=torch.uint8, device=DEV)
        c.reduce_residual_rmsnorm_backward(dys, h, w, 1e-6, dres, dx, dw, workspace=ws)
        c.sync()
    backward.check(dx, dw, dys, h, w, 1e-6, dres, dtype)
    out.check()
