"""Rank sum, global norm and clipping of many gradient tensors (car_grads_*) against plain sums in 64 bits.

Sums and their rounding are exact (fp32 in rank order, one product with the scale).  The norm: at most 64 squares in
a thread and then 32 threads' sums in five levels are added in fp32 (70 roundings of 2^-24 with the square's own), the
rest in 64 bits; the root halves that: 35 * 2^-24, under 2^-18 with the rounding to fp32.  A clipped value is the stored one times a factor known to 2^-18, rounded."""
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


def make(W, sizes, seed, offsets=None, sigma=1.0):
    """W ranks of tensors [(numel, dtype)]; offsets[t] shifts tensor t of every buffer by that many elements, and
    offsets[t] = (a, b, ...) each rank's by its own."""
    g, ranks, out = gen(seed), [], Guarded()
    off = lambda t, r: 0 if offsets is None else offsets[t] if isinstance(offsets[t], int) else offsets[t][r % len(offsets[t])]  # noqa: E731
    for r in range(W):
        ranks.append([randn(g, (n + off(t, r),), d, sigma)[off(t, r):] for t, (n, d) in enumerate(sizes)])
    outs = [out.empty((n + off(t, 0),), TORCH_DTYPE[d])[off(t, 0):] for t, (n, d) in enumerate(sizes)]
    return ranks, outs, out


def expected(ranks, scale):
    """(fp32 sums, norm in 64 bits)."""
    scale = torch.tensor(scale, dtype=torch.float32, device=DEV)
    G = [rank_sum([ranks[r][t] for r in range(len(ranks))]) * scale for t in range(len(ranks[0]))]
    return G, math.sqrt(sum(float((v.double() ** 2).sum()) for v in G))


def check(outs, G, norm, max_norm, got_norm, dtypes):
    assert abs(got_norm - norm) <= NORM_REL * norm
    factor = min(1.0, max_norm / (norm + 1e-6))
    for t, (o, v, d) in enumerate(zip(outs, G, dtypes)):
        stored = v.to(o.dtype)
        if factor == 1.0:
            assert torch.equal(o, stored), f"tensor {t}"
        else:
            want = stored.double() * factor
            assert_within(o, want, (half(d) + NORM_REL) * want.abs() + TINY[d], f"tensor {t}")


BF, HF, FP = "bf16", "fp16", "fp32"
CASES = [
    # (W, [(numel, type)], offsets)
    (1, [(1, BF)], None), (2, [(8, BF), (1, FP), (7, HF)], None), (3, [(0, BF), (5, FP), (0, FP), (4096, BF)], None),
    (4, [(100003, BF), (17, FP), (32769, HF)], [1, 3, 5]), (8, [(16384, BF), (16385, BF), (70001, BF)], [0, 7, 2]),
    (16, [(4099, FP), (333, HF)], [1, 0]), (5, [(2000, BF)] * 40, None), (2, [(3, BF), (9, BF), (31, HF)], [5, 1, 7]),
    (1, [(300001, FP)], [3]), (2, [(1 << 22, BF), (12345, FP)], None),
    # pointers that share no 16-byte boundary: element by element
    (2, [(10007, BF), (555, FP), (2049, HF)], [(0, 1), (1, 2), (3, 4)]), (8, [(5000, BF)], [(0, 1, 2, 3, 4, 5, 6, 7)]),
]


@pytest.mark.parametrize("W,sizes,offsets", CASES)
@pytest.mark.parametrize("max_norm", [math.inf, 0.5, 0.0])
def test_reduce_clip(car, W, sizes, offsets, max_norm):
    ranks, outs, guards = make(W, sizes, seed=len(sizes) + W, offsets=offsets)
    G, norm = expected(ranks, 1.0 / W)
    nbuf = guards.empty((1,), torch.float32)
    with car.Grads(ranks, outs) as g:
        for _ in range(2):  # a second call finds the scratch as the first did
            g.reduce_clip(1.0 / W, max_norm, nbuf)
            torch.cuda.synchronize()
            check(outs, G, norm, max_norm, nbuf.item(), [d for _, d in sizes])
    guards.check()


def test_halves_over_two_handles(car):
    """Two handles of one model: their sums of squares added, both clipped by the total."""
    parts = [make(2, [(5001, BF), (64, FP)], seed=5), make(2, [(70000, HF)], seed=6)]
    exp = [expected(p[0], 0.5) for p in parts]
    norm = math.hypot(exp[0][1], exp[1][1])
    gs = [car.Grads(p[0], p[1]) for p in parts]
    sumsq = torch.empty(2, dtype=torch.float64, device=DEV)
    for k, g in enumerate(gs):
        g.reduce(0.5, sumsq[k:k + 1])
    total = sumsq.sum().reshape(1)
    nb = torch.empty(1, device=DEV)
    for k, (g, p) in enumerate(zip(gs, parts)):
        g.clip(total, 1.0, nb if k else None)
    torch.cuda.synchronize()
    check(parts[0][1], exp[0][0], norm, 1.0, nb.item(), [BF, FP])
    check(parts[1][1], exp[1][0], norm, 1.0, nb.item(), [HF])
    for g in gs:
        g.close()


@pytest.mark.parametrize("rank", [0, 2])
def test_in_place(car, rank):
    ranks, _, _ = make(3, [(4097, BF), (100, FP), (70000, BF)], seed=9)
    G, norm = expected(ranks, 1.0)
    nb = torch.empty(1, device=DEV)
    with car.Grads(ranks, ranks[rank]) as g:
        g.reduce_clip(1.0, 2.0, nb)
        torch.cuda.synchronize()
    check(ranks[rank], G, norm, 2.0, nb.item(), [BF, FP, BF])


def test_one_rank_in_place_is_plain_clipping(car):
    ranks, _, _ = make(1, [(4097, BF), (100, FP), (3, HF)], seed=10)
    G, norm = expected(ranks, 1.0)
    nb = torch.empty(1, device=DEV)
    with car.Grads(ranks, ranks[0]) as g:
        g.reduce_clip(1.0, 1e9, nb)
        torch.cuda.synchronize()
        check(ranks[0], G, norm, 1e9, nb.item(), [BF, FP, HF])
        g.reduce_clip(1.0, norm / 3, nb)
        torch.cuda.synchronize()
    check(ranks[0], G, norm, norm / 3, nb.item(), [BF, FP, HF])


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_values_that_are_not_finite(car, bad):
    ranks, outs, _ = make(2, [(1000, BF), (50, FP)], seed=11)
    ranks[1][1][7] = bad
    nb = torch.empty(1, device=DEV)
    with car.Grads(ranks, outs) as g:
        g.reduce_clip(1.0, 1.0, nb)
        torch.cuda.synchronize()
        if math.isnan(bad):   # a NaN norm reaches every value
            assert math.isnan(nb.item()) and all(o.isnan().all() for o in outs)
        else:                 # an infinite one clips to 0, and 0 * inf is NaN
            assert math.isinf(nb.item()) and (outs[0] == 0).all()
            assert outs[1][7].isnan() and (outs[1][:7] == 0).all()
        g.reduce_clip(1.0, math.inf, nb)
        torch.cuda.synchronize()
        G, _ = expected(ranks, 1.0)   # no limit: the sums, whatever the norm
        assert torch.equal(outs[0], G[0].bfloat16()) and torch.equal(outs[1].nan_to_num(5.0), G[1].nan_to_num(5.0))


def test_large_and_small_tensors_many_chunks_per_cta(car):
    """More chunks than CTAs, sums of squares over 2^25 values: every value and the norm."""
    sizes = [((1 << 25) + 3, BF), (7, BF), ((1 << 24) + 1, FP)]
    ranks, outs, guards = make(2, sizes, seed=12, offsets=[3, 0, 1], sigma=0.01)
    G, norm = expected(ranks, 0.5)
    nb = torch.empty(1, device=DEV)
    with car.Grads(ranks, outs) as g:
        g.reduce_clip(0.5, 1.0, nb)
        torch.cuda.synchronize()
    check(outs, G, norm, 1.0, nb.item(), [BF, BF, FP])
    guards.check()


def test_captured_and_replayed_same_bits(car):
    ranks, outs, _ = make(4, [(100001, BF), (2048, FP)], seed=13)
    nb = torch.empty(1, device=DEV)
    with car.Grads(ranks, outs) as g:
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            g.reduce_clip(0.25, 1.0, nb)
        for seed in (14, 15):
            new, _, _ = make(4, [(100001, BF), (2048, FP)], seed=seed)
            for r in range(4):
                for a, b in zip(ranks[r], new[r]):
                    a.copy_(b)
            G, norm = expected(ranks, 0.25)
            graph.replay()
            torch.cuda.synchronize()
            check(outs, G, norm, 1.0, nb.item(), [BF, FP])
            first = [o.clone() for o in outs], nb.clone()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(first[0], outs)) and torch.equal(first[1], nb)
        del graph


def test_refusals(car):
    ranks, outs, _ = make(2, [(64, BF), (64, FP)], seed=16)
    with pytest.raises(ValueError):
        car.Grads(ranks, outs[:1])
    with pytest.raises(ValueError):
        car.Grads(ranks, [outs[0], outs[1][:63]])
    with pytest.raises(ValueError):
        car.Grads(ranks, [outs[0].half(), outs[1]])
    with pytest.raises(ValueError):
        car.Grads([], outs)
    with pytest.raises(ValueError):
        car.Grads([[x[::2] for x in r] for r in ranks], [o[::2] for o in outs])
    with pytest.raises(ValueError, match="overlap"):
        car.Grads([[r[0], r[0]] for r in ranks], [outs[0], outs[0]])
    with pytest.raises(ValueError, match="overlaps"):
        car.Grads([[ranks[0][0][:32], ranks[0][0][32:]], [ranks[1][0][:32], ranks[1][0][32:]]],
                  [ranks[0][0][16:48], outs[0][:32]])
    with car.Grads(ranks, outs) as g:
        s, nb = torch.empty(1, dtype=torch.float64, device=DEV), torch.empty(1, device=DEV)
        for call in (lambda: g.reduce(math.nan, s), lambda: g.reduce(math.inf, s), lambda: g.clip(s, -1.0),
                     lambda: g.clip(s, math.nan), lambda: g.reduce_clip(math.nan, 1.0)):
            with pytest.raises(car.CarError) as e:
                call()
            assert e.value.status == car.CAR_ERR_ARG
        with pytest.raises(ValueError):
            g.reduce(1.0, nb)
        with pytest.raises(ValueError):
            g.clip(s, 1.0, s)
        assert car.car_grads_reduce(g.h, 1.0, None) == car.CAR_ERR_ARG
        assert car.car_grads_reduce(g.h, 1.0, s.data_ptr() + 4) == car.CAR_ERR_ALIGN
        assert car.car_grads_clip(g.h, s.data_ptr(), 1.0, nb.data_ptr() + 2) == car.CAR_ERR_ALIGN
        h = g.h
    assert car.car_grads_reduce_clip(h, 1.0, 1.0, None) == car.CAR_ERR_HANDLE


def test_norm_over_the_range_of_doubles(car):
    """The root of a caller's sum: in fp32 with 2^-23 to lose (the mantissa's conversion, halved by the root, and the
    root's own rounding), infinite or zero past its range, NaN for what has no root."""
    out = torch.ones(8, device=DEV)
    nb = torch.empty(1, device=DEV)
    with car.Grads([[out]], [out]) as g:
        for value in (0.0, -0.0, 5e-324, 2.0**-1040, 1e-90, 1e-77, 0.1, 1.0, 2.0, 3.0, 3.7e10, 1e70, 1.1e77, 1e80, 1e300, math.inf,
                      math.nan, -1.0, -math.inf):
            g.clip(torch.tensor([value], dtype=torch.float64, device=DEV), math.inf, nb)
            got = nb.item()
            if math.isnan(value) or value < 0:
                assert math.isnan(got), value
                continue
            want = math.sqrt(value)
            if want > 3.4028235677973366e38:  # rounds past the largest fp32
                assert got == math.inf, value
            else:
                assert abs(got - want) <= 2.0**-23 * want + 2.0**-149, (value, got)


@pytest.mark.parametrize("W,n,value", [(1, 1 << 22, 1e18), (2, 3_000_001, 5e17), (1, 1 << 22, 1e-18), (4, 777, 3e-20)])
def test_sums_of_squares_past_the_range_of_fp32(car, W, n, value):
    """Sums above fp32's largest value and squares near its smallest normal ones, over many CTAs: 2^-17 for the squares
    in fp32 (their bound doubled: no root here) and the partials' sum within 2^-41."""
    xs = [torch.full((n,), value, device=DEV) for _ in range(W)]
    out = torch.empty(n, device=DEV)
    sq, nb = torch.empty(1, dtype=torch.float64, device=DEV), torch.empty(1, device=DEV)
    G = xs[0].clone()
    for x in xs[1:]:
        G += x
    want = (G.double() ** 2).sum().item()
    with car.Grads([[x] for x in xs], [out]) as g:
        g.reduce(1.0, sq)
        assert abs(sq.item() - want) <= 2.0**-17 * want
        g.reduce_clip(1.0, math.inf, nb)
        assert abs(nb.item() - math.sqrt(want)) <= NORM_REL * math.sqrt(want)


def test_partials_of_different_size(car):
    """One large value among CTAs of small ones, and an infinity or NaN in one CTA's part."""
    n = 2_000_003
    x = torch.full((n,), 1e-3, device=DEV)
    sq, out = torch.empty(1, dtype=torch.float64, device=DEV), torch.empty(n, device=DEV)
    with car.Grads([[x]], [out]) as g:
        for at, value in ((1_234_567, 1e15), (n - 1, 1e3), (0, math.inf), (777_777, math.nan)):
            x.fill_(1e-3)
            x[at] = value
            g.reduce(1.0, sq)
            want = (x.double() ** 2).sum().item()
            if math.isfinite(want):
                assert abs(sq.item() - want) <= 2.0**-17 * want
            else:
                assert math.isnan(sq.item()) if math.isnan(want) else sq.item() == want
