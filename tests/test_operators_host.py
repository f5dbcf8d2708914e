"""Host-side checks of the operators next to the rank sum: bad handles, and everything a gradient handle refuses
before it touches CUDA.  No test here launches a kernel."""
import pytest


@pytest.fixture(scope="module")
def car():
    import __graft_entry__

    __graft_entry__.build()
    import rank_sum_reduce_gb300 as car

    return car


def test_calls_on_bad_handles(car):
    bogus = 0x1000
    assert car.car_reduce_residual_rmsnorm_quant(bogus, [16], 16, 16, 1e-6, 0, 16, 16, 16, None, None) == car.CAR_ERR_HANDLE
    assert car.car_reduce_residual_rmsnorm_backward(bogus, [16], 16, 16, 1e-6, None, 16, None, None) == car.CAR_ERR_HANDLE
    assert car.car_quant_scale_bytes(bogus, 0) == 0 and car.car_backward_workspace_bytes(bogus) == 0
    assert car.car_grads_destroy(bogus) == car.CAR_ERR_HANDLE and car.car_grads_destroy(None) == car.CAR_ERR_HANDLE
    assert car.car_grads_reduce(bogus, 1.0, 16) == car.CAR_ERR_HANDLE
    assert car.car_grads_clip(bogus, 16, 1.0, None) == car.CAR_ERR_HANDLE
    assert car.car_grads_reduce_clip(bogus, 1.0, 1.0, None) == car.CAR_ERR_HANDLE


def test_pointer_tables_take_what_ctypes_takes(car):
    """Addresses of any integer type, wrapped into 64 bits; nothing else."""
    import numpy as np

    assert car.car_reduce(0x1000, [np.uint64(16), -16, 2**64 + 16, 16.0], 16) == car.CAR_ERR_HANDLE
    with pytest.raises(TypeError):
        car.car_reduce(0x1000, [16, None], 16)


def test_grads_create_refuses_a_total_past_64_bits(car):
    """2^18 tensors of 2^48 fp32 values: 2^64 vectors of 16 bytes, which must not wrap to a small number."""
    n = 2**18
    outs = [(t + 1) << 40 for t in range(n)]
    st, h = car.car_grads_create(1, [2**48] * n, [2] * n, outs, outs)
    assert st == car.CAR_ERR_SIZE and h is None


BF16, FP32 = 0, 2
A, B, C = 0x10000, 0x20000, 0x30000


@pytest.mark.parametrize("W,numel,dtypes,inputs,outs,want", [
    (0, [8], [BF16], [], [C], "ARG"), (17, [8], [BF16], [A] * 17, [C], "ARG"),
    (1, [-1], [BF16], [A], [C], "ARG"), (1, [8], [7], [A], [C], "ARG"), (1, [8], [-1], [A], [C], "ARG"),
    (1, [2**60], [BF16], [A], [C], "SIZE"), (1, [2**48], [BF16], [A], [A], "SIZE"),
    (1, [8], [BF16], None, [C], "ARG"), (1, [8], [BF16], [A], None, "ARG"),
    (1, [8], [BF16], [0], [C], "ARG"), (1, [8], [BF16], [A], [0], "ARG"),
    (1, [8], [BF16], [A + 1], [C], "ALIGN"), (1, [8], [FP32], [A + 2], [C], "ALIGN"), (1, [8], [FP32], [A], [C + 2], "ALIGN"),
    (1, [8, 8], [BF16, BF16], [A, B], [C, C], "ARG"),            # the same output twice
    (1, [8, 8], [BF16, BF16], [A, B], [C, C + 14], "ARG"),       # outputs one element into one another
    (1, [8], [BF16], [A], [A + 2], "ARG"),                       # an output one element into its input
    (2, [8, 8], [BF16, BF16], [A, B, A + 64, B + 64], [B, A], "ARG"),   # each other's input
    (1, [100, 8], [BF16, BF16], [A, A + 400], [A, A + 100], "ARG"),     # inside another tensor's input and output
])
def test_grads_create_refuses(car, W, numel, dtypes, inputs, outs, want):
    st, h = car.car_grads_create(W, numel, dtypes, inputs, outs)
    assert st == getattr(car, "CAR_ERR_" + want) and h is None


@pytest.mark.parametrize("W,numel,inputs,outs", [
    (1, [8, 8], [A, A + 16], [A, A + 16]),            # in place, neighbours
    (2, [8, 0], [A, 0, A, 0], [C, 0]),                # the same buffer for two ranks; an empty tensor
    (2, [8, 8], [A, B, A + 16, B + 16], [A + 16, B]),  # each in place of another rank
    (1, [8], [A], [A + 16]),                          # behind its input
])
def test_grads_create_accepts(car, W, numel, inputs, outs):
    """Past its own checks; without a GPU the CUDA runtime then says so."""
    import torch

    if torch.cuda.is_available():
        pytest.skip("addresses are made up")
    st, h = car.car_grads_create(W, numel, [BF16] * len(numel), inputs, outs)
    assert st == car.CAR_ERR_CUDA and h is None and car.car_last_error()
