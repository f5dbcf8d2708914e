"""Gradient sums past the range of their type, between the two passes of car_grads_reduce_clip and in car_grads_reduce.

Against the definition in 64 bits, G * min(1, max_norm / (norm + 1e-6)).  A value of two and more ranks is rounded twice,
once as a sum and once clipped, each time by half(t) relative or TINY; the factor is known to 2^-18 as in the other
tests of the norm: (2 half + half^2 + 2^-18) |want| + 2 TINY.  The first term is 2.01 half + 2^-18 for every type here."""
import math

import pytest
import torch

from operator_checks import DEV, TINY, TORCH_DTYPE, Guarded, assert_within, gen, half, randn, rank_sum

pytestmark = pytest.mark.gpu
NORM_REL = 2.0**-18
BF, HF, FP = "bf16", "fp16", "fp32"


@pytest.fixture(scope="module")
def car():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import rank_sum_reduce_gb300 as car

    return car


def make(W, sizes, offsets, seed):
    """Ranks of tensors [(numel, dtype)], tensor t of rank r from element offsets[t][r] of its buffer (the output from
    offsets[t][0]); every fifth value of a 16-bit tensor is 3e4 to 6e4 in every rank, one sign per place."""
    g, ranks, out = gen(seed), [[] for _ in range(W)], Guarded()
    outs = []
    for t, (n, d) in enumerate(sizes):
        off = offsets[t] if offsets else (0,)
        loud = torch.arange(n, device=DEV) % 5 == 2
        sign = torch.where(torch.rand(n, generator=g, device=DEV) < 0.5, -1.0, 1.0)
        for r in range(W):
            raw = torch.empty(n + off[r % len(off)], dtype=TORCH_DTYPE[d], device=DEV)
            x = raw[off[r % len(off)]:]
            x.copy_(randn(g, (n,), FP))
            if d != FP:
                x[loud] = (sign * (3e4 + 3e4 * torch.rand(n, generator=g, device=DEV)))[loud].to(x.dtype)
            ranks[r].append(x)
        outs.append(out.empty((n + off[0],), TORCH_DTYPE[d])[off[0]:])
    return ranks, outs, out


def sums(ranks, scale):
    """(fp32 sums, norm in 64 bits)."""
    scale = torch.tensor(scale, dtype=torch.float32, device=DEV)
    G = [rank_sum([x[t] for x in ranks]) * scale for t in range(len(ranks[0]))]
    return G, math.sqrt(sum(float((v.double() ** 2).sum()) for v in G))


def check(outs, G, norm, max_norm, got):
    assert abs(got - norm) <= NORM_REL * norm
    factor = min(1.0, max_norm / (norm + 1e-6))
    for t, (o, v) in enumerate(zip(outs, G)):
        if factor == 1.0:   # one rounding, to infinity where the sum is past the range
            assert torch.equal(o, v.to(o.dtype)), f"tensor {t}"
            continue
        d = {torch.bfloat16: BF, torch.float16: HF, torch.float32: FP}[o.dtype]
        want = v.double() * factor
        assert_within(o, want, (2.01 * half(d) + NORM_REL) * want.abs() + 2 * TINY[d], f"tensor {t}")


CASES = [
    # (W, tensors, offsets): runtime and compiled rank counts, ragged ends, pointers without a common 16-byte boundary
    (2, [(1, HF), (4096, HF), (100, FP), (4097, BF)], None),
    (3, [(70001, HF)], [(3,)]),
    (4, [(32769, HF), (17, FP)], [(5,), (1,)]),
    (5, [(2000, HF)] * 3, None),
    (6, [(9001, HF), (5000, BF)], [(0,), (7,)]),
    (8, [(16385, HF), (40000, HF)], [(0,), (2,)]),
    (16, [(4099, HF)], [(1,)]),
    (2, [(10007, HF), (2049, HF)], [(0, 1), (3, 4)]),
    (8, [(5000, HF)], [(0, 1, 2, 3, 4, 5, 6, 7)]),
    (2, [(3_000_001, HF)], None),
]


@pytest.mark.parametrize("W,sizes,offsets", CASES)
@pytest.mark.parametrize("place", ["apart", "first", "last"])
def test_sums_past_fp16_are_clipped_into_range(car, W, sizes, offsets, place):
    for max_norm in (1000.0, 0.0, 1e30, math.inf):
        ranks, outs, guards = make(W, sizes, offsets, seed=W + len(sizes))
        G, norm = sums(ranks, 1.0)
        assert max(float(v.abs().max()) for v in G) > 65520 or sizes[0][0] == 1
        outs = {"apart": outs, "first": ranks[0], "last": ranks[-1]}[place]
        nb = torch.empty(1, device=DEV)
        with car.Grads(ranks, outs) as g:
            for _ in range(2 if place == "apart" else 1):
                g.reduce_clip(1.0, max_norm, nb)
                torch.cuda.synchronize()
                check(outs, G, norm, max_norm, nb.item())
        guards.check()


@pytest.mark.parametrize("place", ["apart", "in place"])
def test_infinite_and_nan_values_stay_what_they_are(car, place):
    """An infinity of a rank is one of the gradients (its norm clips to 0, and 0 * inf is NaN), and so is a NaN."""
    for bad in (math.inf, math.nan):
        ranks, outs, _ = make(2, [(1000, HF), (64, HF)], None, seed=3)
        ranks[1][0][7] = bad
        outs = outs if place == "apart" else ranks[1]
        nb = torch.empty(1, device=DEV)
        with car.Grads(ranks, outs) as g:
            g.reduce_clip(1.0, 1.0, nb)
            torch.cuda.synchronize()
        if math.isnan(bad):
            assert math.isnan(nb.item()) and all(o.isnan().all() for o in outs)
        else:
            assert math.isinf(nb.item()) and outs[0][7].isnan()
            assert (outs[0][8:] == 0).all() and (outs[0][:7] == 0).all() and (outs[1] == 0).all()


def test_captured_in_place(car):
    """The same list captured once and replayed on new values, in place, within the limit and over it."""
    sizes = [(10001, HF), (333, BF)]
    ranks, _, _ = make(4, sizes, None, seed=1)
    nb = torch.empty(1, device=DEV)
    with car.Grads(ranks, ranks[2]) as g:
        for max_norm in (500.0, 1e30):
            graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=side):
                g.reduce_clip(0.5, max_norm, nb)
            for seed in (5, 6):
                new, _, _ = make(4, sizes, None, seed=seed)
                for r in range(4):
                    for a, b in zip(ranks[r], new[r]):
                        a.copy_(b)
                G, norm = sums(ranks, 0.5)
                graph.replay()
                torch.cuda.synchronize()
                check(ranks[2], G, norm, max_norm, nb.item())
            del graph


@pytest.mark.parametrize("W,offsets", [(1, None), (2, None), (2, [(0, 1), (0, 0)]), (5, None), (8, None)])
@pytest.mark.parametrize("place", ["apart", "in place"])
def test_stored_infinities_count_in_the_sum_of_squares(car, W, offsets, place):
    """car_grads_reduce stores its sums, so one that is infinite in fp16 makes the sum of squares infinite too (it would
    not tell otherwise of what car_grads_clip cannot bring back); 65519 is stored as 65504 and does not."""
    sq = torch.empty(1, dtype=torch.float64, device=DEV)
    for value in (65519.0, 65520.0, -65519.0, -65520.0, 1e18):
        for at in (0, 4001, 4002):   # in a whole vector, in the tail, nowhere
            ranks, outs, _ = make(W, [(4002, HF), (64, FP)], offsets, seed=2)
            scale = 2 * abs(value)   # a half of it is exact
            for r in range(W):
                ranks[r][0].zero_()
                ranks[r][1].div_(scale)
            if at < 4002:
                ranks[-1][0][at] = math.copysign(0.5, value)
            G, norm = sums(ranks, scale)
            outs = outs if place == "apart" else ranks[0]
            with car.Grads(ranks, outs) as g:
                g.reduce(scale, sq)
                torch.cuda.synchronize()
            assert torch.equal(outs[0], G[0].half()) and torch.equal(outs[1], G[1])
            if at < 4002 and abs(value) >= 65520:
                assert outs[0][at].isinf() and sq.item() == math.inf
            else:
                assert outs[0].isfinite().all() and abs(sq.item() - norm**2) <= 2.0**-17 * norm**2


def test_a_nan_is_not_covered_by_an_infinity(car):
    ranks, outs, _ = make(2, [(5000, HF)], None, seed=4)
    ranks[0][0][17], ranks[1][0][4000] = math.nan, 6e4
    sq = torch.empty(1, dtype=torch.float64, device=DEV)
    with car.Grads(ranks, outs) as g:
        g.reduce(4.0, sq)
        torch.cuda.synchronize()
    assert math.isnan(sq.item())
