"""Gradient sums clipped with one rounding (car_grads_reduce_clip_once) against the definition in 64 bits.

G is exact in fp32 (rank order, one product with the scale); a value is G * factor, the factor known to 2^-18 as the norm
is (see test_grads_gpu), rounded once: half(t) |want| + 2^-18 |want| + TINY.  An fp16 value within that of 65520 may be
its largest or infinite."""
import math

import pytest
import torch

from operator_checks import DEV, TINY, TORCH_DTYPE, Guarded, assert_within, gen, half, randn, rank_sum

pytestmark = pytest.mark.gpu
NORM_REL = 2.0**-18


@pytest.fixture(scope="module")
def car():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import rank_sum_reduce_gb300 as car

    return car


# (tensors, first element of each in its buffer, by rank; the output's is the last)
LISTS = [
    ([(40000, "bf16"), (8, "fp16"), (4096, "fp32"), (70001, "fp16")], [(0,), (0,), (0,), (0,)]),
    ([(70003, "fp16"), (33, "fp32"), (20001, "bf16"), (5, "bf16"), (0, "bf16"), (1, "fp16")], [(3,), (1,), (7,), (2,), (0,), (5,)]),
    ([(10007, "bf16"), (2049, "fp16"), (555, "fp32")], [(0, 1, 2), (3, 4), (1, 2)]),   # no common 16-byte boundary
]


def make(W, sizes, offs, seed, sigma=1.0):
    g, out = gen(seed), Guarded()
    ranks = [[randn(g, (n + o[r % len(o)],), d, sigma)[o[r % len(o)]:] for (n, d), o in zip(sizes, offs)] for r in range(W)]
    return ranks, [out.empty((n + o[-1],), TORCH_DTYPE[d])[o[-1]:] for (n, d), o in zip(sizes, offs)], out


def sums(ranks, scale):
    f = torch.tensor(scale, dtype=torch.float32, device=DEV)
    G = [rank_sum([x[t] for x in ranks]) * f for t in range(len(ranks[0]))]
    return G, math.sqrt(sum(float((v.double() ** 2).sum()) for v in G))


def check(outs, G, sizes, norm, max_norm, got):
    assert abs(got - norm) <= NORM_REL * norm
    factor = min(1.0, max_norm / (norm + 1e-6))
    for t, (o, v, (_, d)) in enumerate(zip(outs, G, sizes)):
        if factor == 1.0:
            assert torch.equal(o, v.to(o.dtype)), f"tensor {t}"
            continue
        want = v.double() * factor
        room = (half(d) + NORM_REL) * want.abs() + TINY[d]
        if d == "fp16":
            past = want.abs() - 65520
            assert (o[past > room] == torch.sign(want[past > room]) * math.inf).all()
            o, want, room = o[past < -room], want[past < -room], room[past < -room]
        assert_within(o, want, room, f"tensor {t}")


@pytest.mark.parametrize("W", [1, 2, 3, 4, 5, 8, 12, 16])
@pytest.mark.parametrize("sizes,offs", LISTS)
@pytest.mark.parametrize("place", ["apart", "in place"])
def test_matches_definition(car, W, sizes, offs, place):
    nb = torch.empty(1, device=DEV)
    for scale, limit in ((1.0, 0.25), (1.0 / 3, 0.9), (1.0 / W, 2.0), (0.5, 0.0), (1.0, math.inf)):
        ranks, outs, guards = make(W, sizes, offs, seed=W)
        G, norm = sums(ranks, scale)
        outs = outs if place == "apart" else ranks[W // 2]
        with car.Grads(ranks, outs) as g:
            for _ in range(2 if place == "apart" else 1):
                g.reduce_clip(scale, limit * norm, nb, once=True)
                torch.cuda.synchronize()
                check(outs, G, sizes, norm, limit * norm, nb.item())
        guards.check()


@pytest.mark.parametrize("place", ["apart", "in place"])
def test_one_rounding_is_nearer_than_two(car, place):
    """The mean error of many values: a rounding's is eps / 4 / sqrt(3) relative at most, two give 1.41 times that
    where the factor is no power of two; half way between is 1.2."""
    sizes = [(1 << 20, "bf16"), (1 << 20, "fp16")]
    nb = torch.empty(1, device=DEV)
    err = {}
    for once in (False, True):
        ranks, outs, _ = make(4, sizes, [(0,), (0,)], seed=8)
        G, norm = sums(ranks, 0.25)
        outs = outs if place == "apart" else ranks[0]
        with car.Grads(ranks, outs) as g:
            g.reduce_clip(0.25, norm / 3, nb, once=once)
            torch.cuda.synchronize()
        err[once] = [float((o.double() - v.double() / 3).norm() / (v.double() / 3).norm()) for o, v in zip(outs, G)]
    for two, one, (_, d) in zip(err[False], err[True], sizes):
        assert one <= 0.5 * torch.finfo(TORCH_DTYPE[d]).eps / 3**0.5 and two > 1.2 * one


@pytest.mark.parametrize("place", ["apart", "in place"])
def test_sums_past_fp16(car, place):
    sizes = [(70001, "fp16"), (300, "bf16")]
    nb = torch.empty(1, device=DEV)
    for W, max_norm in ((2, 1000.0), (7, 1e30), (16, 5e6)):
        ranks, outs, _ = make(W, sizes, [(1,), (0,)], seed=W, sigma=2e4)
        for r in ranks:
            r[0].clamp_(-65504, 65504)
        G, norm = sums(ranks, 1.0)
        assert float(G[0].abs().max()) > 65520
        outs = outs if place == "apart" else ranks[-1]
        with car.Grads(ranks, outs) as g:
            g.reduce_clip(1.0, max_norm, nb, once=True)
            torch.cuda.synchronize()
        check(outs, G, sizes, norm, max_norm, nb.item())


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_values_that_are_not_finite(car, bad):
    ranks, outs, _ = make(2, [(1000, "bf16"), (50, "fp32"), (64, "fp16")], [(0,)] * 3, seed=11)
    ranks[1][0][7] = bad
    nb = torch.empty(1, device=DEV)
    with car.Grads(ranks, outs) as g:
        g.reduce_clip(1.0, 1.0, nb, once=True)
        torch.cuda.synchronize()
    if math.isnan(bad):
        assert math.isnan(nb.item()) and all(o.isnan().all() for o in outs)
    else:
        assert math.isinf(nb.item()) and outs[0][7].isnan() and (outs[0][8:] == 0).all() and (outs[1] == 0).all()


@pytest.mark.parametrize("place", ["apart", "in place"])
def test_captured_and_replayed_same_bits(car, place):
    sizes = [(100001, "bf16"), (2048, "fp32"), (999, "fp16")]
    ranks, outs, _ = make(4, sizes, [(0,)] * 3, seed=13)
    outs = outs if place == "apart" else ranks[3]
    nb = torch.empty(1, device=DEV)
    with car.Grads(ranks, outs) as g:
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            g.reduce_clip(0.25, 1.0, nb, once=True)
        first = None
        for _ in range(2):
            new, _, _ = make(4, sizes, [(0,)] * 3, seed=14)
            for r in range(4):
                for a, b in zip(ranks[r], new[r]):
                    a.copy_(b)
            G, norm = sums(ranks, 0.25)
            graph.replay()
            torch.cuda.synchronize()
            check(outs, G, sizes, norm, 1.0, nb.item())
            if first is not None:
                assert all(torch.equal(a, b) for a, b in zip(first, outs))
            first = [o.clone() for o in outs]
        del graph
