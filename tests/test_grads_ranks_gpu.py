"""Gradient sums of every rank count, each output: the sums alone (car_grads_reduce), the sums within the limit and over
it, apart from the inputs and in place of one.

Sums and their rounding are exact (fp32 in rank order, one product with the scale), the norm lies within 2^-18 and the
sum of squares within 2^-17 (see test_grads_gpu).  A clipped value of one rank is G * factor rounded once, of more the
stored sum * factor, rounded: half(t) and the factor's 2^-18."""
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


# (tensors, first element of each in its buffer): whole vectors and ragged ends, chunks of more than one pass
LISTS = [([(40000, "bf16"), (8, "fp16"), (4096, "fp32")], (0, 0, 0)),
         ([(70003, "fp16"), (33, "fp32"), (20001, "bf16"), (5, "bf16")], (3, 1, 7, 2))]


def make(W, sizes, offs, seed):
    g, out = gen(seed), Guarded()
    ranks = [[randn(g, (n + o,), d)[o:] for (n, d), o in zip(sizes, offs)] for _ in range(W)]
    return ranks, [out.empty((n + o,), TORCH_DTYPE[d])[o:] for (n, d), o in zip(sizes, offs)], out


@pytest.mark.parametrize("W", range(1, 17))
@pytest.mark.parametrize("sizes,offs", LISTS)
@pytest.mark.parametrize("place", ["apart", "in place"])
@pytest.mark.parametrize("scale", [1.0, 1.0 / 3])
def test_sums_and_clipped_sums(car, W, sizes, offs, place, scale):
    sq, nb = torch.empty(1, dtype=torch.float64, device=DEV), torch.empty(1, device=DEV)
    for limit in (None, 2.0, 0.25, 0.0):   # alone; twice the norm, a quarter of it, nothing
        ranks, outs, guards = make(W, sizes, offs, seed=W)
        f = torch.tensor(scale, dtype=torch.float32, device=DEV)
        G = [rank_sum([x[t] for x in ranks]) * f for t in range(len(sizes))]
        norm = math.sqrt(sum(float((v.double() ** 2).sum()) for v in G))
        outs = outs if place == "apart" else ranks[W // 2]
        with car.Grads(ranks, outs) as g:
            if limit is None:
                g.reduce(scale, sq)
            else:
                g.reduce_clip(scale, limit * norm, nb)
            torch.cuda.synchronize()
        if limit is None:
            assert abs(sq.item() - norm**2) <= 2.0**-17 * norm**2
        else:
            assert abs(nb.item() - norm) <= NORM_REL * norm
        guards.check()
        factor = 1.0 if limit is None else min(1.0, limit * norm / (norm + 1e-6))
        for t, (o, v) in enumerate(zip(outs, G)):
            d = sizes[t][1]
            if factor == 1.0:
                assert torch.equal(o, v.to(o.dtype)), f"tensor {t}"
            else:
                want = (v if W == 1 else v.to(o.dtype)).double() * factor
                assert_within(o, want, (half(d) + NORM_REL) * want.abs() + TINY[d], f"tensor {t}")
