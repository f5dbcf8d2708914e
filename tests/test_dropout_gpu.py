"""Dropout of the rank sum (car_reduce_dropout): the mask bit for bit against the generator in numpy, values, edges of p,
offsets on the device, in place, captured, refusals.  A kept value is the exact fp32 rank sum times a factor rounded to
fp32, rounded once more to fp32 and then to the type: 2^-23 and half a step, relative."""
import pytest
import torch

from branch_checks import factor, threshold
from operator_checks import DEV, TINY, TORCH_DTYPE, Guarded, assert_within, gen, half, randn, rank_sum

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def car():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import rank_sum_reduce_gb300 as car

    return car


def check(out, xs, f, dtype):
    want = rank_sum(xs).double() * f
    assert_within(out, want, half(dtype) * want.abs() + 2.0**-22 * want.abs() + TINY[dtype], "dropout")
    assert ((out == 0) | (f != 0)).all()


SHAPES = [(1, 1, 8, "bf16"), (1, 1, 4, "fp32"), (2, 61, 1032, "bf16"), (3, 7, 1000, "fp16"), (4, 33, 132, "fp32"),
          (8, 300, 4096, "bf16"), (16, 5, 2056, "fp16"), (5, 1, 65544, "bf16"), (8, 9, 20, "fp32"), (2, 4099, 2048, "fp16"),
          (1, 2000, 4104, "bf16"), (16, 1, 4, "fp32"), (4, 1001, 1028, "fp32")]


@pytest.mark.parametrize("W,M,N,dtype", SHAPES)
@pytest.mark.parametrize("p", [0.1, 0.5])
def test_matches_the_generator(car, W, M, N, dtype, p):
    g = gen(W + M + N)
    xs = [randn(g, (M, N), dtype) + 4 for _ in range(W)]  # few zeros: what is 0 was dropped, or was 0
    out = Guarded()
    to = out.empty((M, N), TORCH_DTYPE[dtype])
    seed, offset = 2**64 - 5 * W, 2**50 + M
    with car.Car(W, M, N, dtype) as c:
        c.reduce_dropout(xs, car.Dropout(p, seed, offset), to)
        c.sync()
    f = factor(M, N, p, seed, offset)
    assert torch.equal(to == 0, (f == 0) | (rank_sum(xs) == 0))
    check(to, xs, f, dtype)
    out.check()


def test_mask_is_the_same_for_every_type_and_rank_count(car):
    M, N, drop = 37, 264, car.Dropout(0.3, 99, 5)
    masks = []
    for W, dtype in ((1, "bf16"), (8, "fp16"), (3, "fp32")):
        xs, out = [torch.ones(M, N, device=DEV).to(TORCH_DTYPE[dtype]) for _ in range(W)], torch.empty(M, N, device=DEV)
        out = out.to(TORCH_DTYPE[dtype])
        with car.Car(W, M, N, dtype) as c:
            c.reduce_dropout(xs, drop, out)
            c.sync()
        masks.append(out == 0)
    assert torch.equal(masks[0], masks[1]) and torch.equal(masks[0], masks[2]) and masks[0].any() and not masks[0].all()


def test_nothing_and_everything_dropped(car):
    W, M, N = 2, 19, 520
    g = gen(1)
    xs, out, plain = [randn(g, (M, N), "bf16") for _ in range(W)], *(torch.empty(M, N, device=DEV).bfloat16() for _ in range(2))
    with car.Car(W, M, N, "bf16") as c:
        c.reduce(xs, plain)
        for p in (0.0, 2.0**-18):
            c.reduce_dropout(xs, car.Dropout(p, 3), out)
            c.sync()
            assert torch.equal(out, plain)
        xs[0][0] = float("nan")
        xs[1][1] = float("inf")
        c.reduce_dropout(xs, car.Dropout(1.0, 3), out)
        c.sync()
        assert (out == 0).all()
        p = 65535 / 65536           # one value in 65536 is kept, times 65536
        c.reduce_dropout(xs, car.Dropout(p, 3), out)
        c.sync()
        f = factor(M, N, p, 3, 0)
        assert threshold(p) == 65535 and torch.equal(out[2:] == 0, (f * rank_sum(xs).double())[2:] == 0)


def test_dropped_infinities_and_nan_are_zero(car):
    W, M, N = 3, 64, 256
    xs = [torch.full((M, N), v, device=DEV) for v in (float("inf"), 1.0, float("nan"))]
    out = torch.empty(M, N, device=DEV)
    with car.Car(W, M, N, "fp32") as c:
        c.reduce_dropout(xs, car.Dropout(0.5, 8, 8), out)
        c.sync()
    f = factor(M, N, 0.5, 8, 8)
    assert (out[f == 0] == 0).all() and out[f != 0].isnan().all()


def test_in_place_of_one_rank(car):
    W, M, N = 4, 77, 1032
    g = gen(5)
    xs = [randn(g, (M, N), "fp16") for _ in range(W)]
    keep = [x.clone() for x in xs]
    with car.Car(W, M, N, "fp16") as c:
        c.reduce_dropout(xs, car.Dropout(0.25, 1, 2), xs[2])
        c.sync()
    check(xs[2], keep, factor(M, N, 0.25, 1, 2), "fp16")


def test_gradient_is_the_same_call(car):
    """Against the forward's own differences: the call is linear, so <out(x), g> = <x_r, dx> for every rank."""
    W, M, N = 3, 21, 260
    g, drop = gen(6), car.Dropout(0.2, 11, 12)
    x, dys = randn(g, (M, N), "fp32"), [randn(g, (M, N), "fp32") for _ in range(W)]
    out, dx = torch.empty_like(x), torch.empty_like(x)
    with car.Car(1, M, N, "fp32") as c, car.Car(W, M, N, "fp32") as cw:
        c.reduce_dropout([x], drop, out)
        cw.reduce_dropout(dys, drop, dx)
        cw.sync()
    lhs, rhs = (out.double() * rank_sum(dys).double()), (x.double() * dx.double())
    assert abs(lhs.sum() - rhs.sum()) <= 2.0**-21 * lhs.abs().sum()


def test_offset_on_the_device_in_a_replayed_graph(car):
    """Also the first use of the call on a handle, inside the capture."""
    W, M, N = 2, 50, 1024
    g = gen(7)
    xs, out = [randn(g, (M, N), "bf16") + 4 for _ in range(W)], torch.empty(M, N, device=DEV).bfloat16()
    step = torch.zeros(1, dtype=torch.int64, device=DEV)
    drop = car.Dropout(0.4, 21, 2**64 - 1, offset_dev=step)   # the sum wraps
    with car.Car(W, M, N, "bf16") as c:
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            c.reduce_dropout(xs, drop, out)
            step.add_(1)
        for k in range(3):
            graph.replay()
            c.sync()
            check(out, xs, factor(M, N, 0.4, 21, (2**64 - 1 + k) % 2**64), "bf16")
        del graph


def test_offsets_past_32_bits_of_elements(car):
    """4.3 billion elements: the counter is the element's place in 64 bits."""
    M, N = 2**20 + 3, 4096
    x = torch.ones(M, N, device=DEV, dtype=torch.bfloat16)
    with car.Car(1, M, N, "bf16") as c:
        c.reduce_dropout([x], car.Dropout(0.5, 77, 3), x)
        c.sync()
    last = x[2**20:]
    at = torch.arange(2**20 * N // 8, M * N // 8)
    import numpy as np

    from branch_checks import philox

    words = np.zeros((at.numel(), 4), dtype=np.uint64)
    words[:, 0], words[:, 1], words[:, 2] = at.numpy() % 2**32, at.numpy() // 2**32, 3
    w = philox(words, (77, 0))
    bits = np.stack([w & 0xFFFF, w >> 16], 2).reshape(3, N)
    assert torch.equal(last.float().cpu(), torch.from_numpy((bits >= 32768) * 2.0).float())


def test_refusals(car):
    W, M, N = 2, 4, 64
    g = gen(1)
    xs, out = [randn(g, (M, N), "bf16") for _ in range(W)], torch.empty(M, N, device=DEV).bfloat16()
    with car.Car(W, M, N, "bf16") as c:
        P = [x.data_ptr() for x in xs]
        drop = lambda p, dev=None: car.car_dropout(p, 1, 2, dev)  # noqa: E731
        for p in (-0.1, 1.01, float("nan"), float("inf")):
            assert car.car_reduce_dropout(c.h, P, drop(p), out.data_ptr()) == car.CAR_ERR_ARG
        assert car.car_reduce_dropout(c.h, P, None, out.data_ptr()) == car.CAR_ERR_ARG
        assert car.car_reduce_dropout(c.h, None, drop(0.1), out.data_ptr()) == car.CAR_ERR_ARG
        assert car.car_reduce_dropout(c.h, P, drop(0.1), None) == car.CAR_ERR_ARG
        assert car.car_reduce_dropout(c.h, P, drop(0.1), out.data_ptr() + 2) == car.CAR_ERR_ALIGN
        assert car.car_reduce_dropout(c.h, P, drop(0.1, 4), out.data_ptr()) == car.CAR_ERR_ALIGN
        with pytest.raises(ValueError):
            c.reduce_dropout(xs, car.Dropout(0.1, 1), out[:-1])
        with pytest.raises(ValueError):
            c.reduce_dropout(xs[:1], car.Dropout(0.1, 1), out)
