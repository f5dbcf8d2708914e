"""Host-side checks of dropout and of a block's branch: the generator's published test vectors, bad handles, and what the
binding refuses before any pointer is taken.  No test here launches a kernel."""
import numpy as np
import pytest


@pytest.fixture(scope="module")
def car():
    import __graft_entry__

    __graft_entry__.build()
    import rank_sum_reduce_gb300 as car

    return car


@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_generator_of_the_tests_gives_the_published_vectors(counter, key, want):
    from branch_checks import philox

    assert philox(np.array([counter], dtype=np.uint64), key).tolist() == [list(want)]


def test_mask_of_the_tests_has_its_rate_and_mean():
    """A million elements at p = 0.1: the dropped count is within 6 deviations of its mean, sqrt(n p (1 - p)) = 300."""
    from branch_checks import factor, threshold

    f = factor(1000, 1000, 0.1, 7, 2**40, device="cpu")
    t = threshold(0.1)
    assert t == 6554
    assert abs(int((f == 0).sum()) - 1e6 * t / 65536) < 6 * 300
    assert set(f.unique().tolist()) == {0.0, 65536 / (65536 - t)}


def test_calls_on_bad_handles(car):
    bogus = 0x1000
    drop, branch, out = car.car_dropout(0.1, 1, 2, None), car.car_branch(), car.car_branch_grads(16)
    assert car.car_reduce_dropout(bogus, [16], drop, 16) == car.CAR_ERR_HANDLE
    assert car.car_reduce_branch_residual_rmsnorm(bogus, [16], branch, 16, 16, 1e-6, 16, 16, None) == car.CAR_ERR_HANDLE
    assert car.car_reduce_branch_residual_rmsnorm_backward(bogus, [16], branch, 16, 16, 16, 1e-6, None, out,
                                                           None) == car.CAR_ERR_HANDLE
    assert car.car_branch_workspace_bytes(bogus, branch) == 0 and car.car_branch_workspace_bytes(None, None) == 0


@pytest.mark.parametrize("p", [-0.1, 1.5, float("nan"), float("inf")])
def test_dropout_refuses_other_probabilities(car, p):
    with pytest.raises(ValueError, match="p: "):
        car.Dropout(p, 0)


def test_dropout_takes_any_seed_and_offset(car):
    d = car.Dropout(0.5, -1, 2**64 + 3)
    assert (d.seed, d.offset) == (2**64 - 1, 3)
    d.seed, d.offset = 2**65 + 9, -2
    assert (d.seed, d.offset, d.struct.seed) == (9, 2**64 - 2, 9)


def test_offset_on_the_device_has_64_bits_and_is_on_the_gpu(car):
    import torch

    with pytest.raises(ValueError, match="offset_dev: torch.int32"):
        car.Dropout(0.1, 0, offset_dev=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        car.Dropout(0.1, 0, offset_dev=torch.zeros(1, dtype=torch.int64))


def test_branch_refuses_negative_gate_rows(car):
    with pytest.raises(ValueError, match="gate_rows"):
        car.Branch(gate_rows=-1)


@pytest.mark.parametrize("name", ["dweight", "dnorm_weight", "dgate"])
@pytest.mark.parametrize("bad", ["bfloat16", "float64", "int64"])
def test_sums_over_rows_of_another_type_are_refused(car, name, bad):
    import torch

    c = object.__new__(car.Car)   # the check needs no handle
    c.h, c.D, c.N = None, 512, 64
    t = torch.empty(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match=f"{name}: torch.{bad}"):
        c.reduce_branch_residual_rmsnorm_backward([t], car.Branch(), t, t, t[0], 1e-6, None, t,
                                                  **{name: torch.empty(64, dtype=getattr(torch, bad))})
