"""Host-side checks of the clipping with one rounding: bad handles.  No test here launches a kernel."""
import pytest


@pytest.fixture(scope="module")
def car():
    import __graft_entry__

    __graft_entry__.build()
    import rank_sum_reduce_gb300 as car

    return car


def test_calls_on_bad_handles(car):
    for bogus in (None, 0x1000):
        assert car.car_grads_reduce_clip_once(bogus, 1.0, 1.0, None) == car.CAR_ERR_HANDLE
