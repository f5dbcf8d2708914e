"""The fused op with an 8-bit output (car_reduce_residual_rmsnorm_quant) against its definition in 64 bits.

The sum and residual_out are exact (fp32 in rank order), scales lie within DELTA of amax / 448, and every code is a
nearest e4m3 value of y / s, with y / s known to within 2 DELTA (see operator_checks)."""
import math

import pytest
import torch

from operator_checks import DELTA, DEV, TINY, TORCH_DTYPE, Guarded, assert_within, gen, half, randn, rank_sum

pytestmark = pytest.mark.gpu
KINDS = ("row", "group128", "mx32", "static")
WIDTH = {"group128": 128, "mx32": 32}


@pytest.fixture(scope="module")
def car():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import rank_sum_reduce_gb300 as car

    return car


def make(W, M, N, dtype, seed):
    g = gen(seed)
    xs = [randn(g, (M, N), dtype) for _ in range(W)]
    res = randn(g, (M, N), dtype) * torch.where(torch.rand(N, generator=g, device=DEV) < 0.02, 20.0, 1.0).to(TORCH_DTYPE[dtype])
    w = (torch.rand(N, generator=g, device=DEV) + 0.5).to(TORCH_DTYPE[dtype])
    return xs, res, w


def normalised(xs, res, w, eps):
    """(h as the kernels form it, y in 64 bits)."""
    h = rank_sum(xs) + res.float()
    d = h.double()
    return h, d * w.double() / torch.sqrt((d * d).mean(1, keepdim=True) + eps)


def scale_values(s):
    return torch.exp2(s.double() - 127) if s.dtype == torch.uint8 else s.double()


def spread(s, width, N):
    return s.repeat_interleave(width, 1)[:, :N]


def check_codes(q, v, what):
    """q is a nearest e4m3 value of v, |v| <= 448 after saturation, v known to within 2 DELTA."""
    v = v.clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0**-6)))) / 8
    assert_within(q, v, step / 2 + 2 * DELTA * v.abs(), what)


def check_scales(kind, s, y):
    M, N = y.shape
    width = WIDTH.get(kind, N)
    pad = torch.nn.functional.pad(y.abs(), (0, -N % width))
    want = (pad.reshape(M, -1, width).amax(2) / 448.0).clamp_min(2.0**-126)
    got = scale_values(s)
    if kind == "mx32":  # the smallest power of two that is not below
        assert (got >= want * (1 - DELTA)).all() and (got / 2 < want * (1 + DELTA)).all()
    else:
        assert_within(got, want, DELTA * want, "scales")
    return spread(got, width, N)


CASES = [
    # (W, M, N, dtype): one CTA per row, one and two vectors per thread, rows split over 4 and 8 CTAs, many rows per
    # CTA, rows shorter than a group, ragged last groups, the longest rows, every compiled rank count and the others
    (1, 1, 8, "bf16"), (1, 5000, 40, "bf16"), (2, 1, 2048, "bf16"), (2, 3, 136, "fp16"), (3, 7, 1000, "bf16"),
    (4, 300, 2056, "bf16"), (4, 160, 8192, "bf16"), (8, 1, 8192, "bf16"), (8, 24, 8200, "bf16"), (8, 700, 4104, "fp16"),
    (16, 2, 4100, "fp32"), (16, 9, 1544, "bf16"), (5, 2, 32768, "bf16"), (2, 4, 16384, "fp32"), (1, 33, 4, "fp32"),
    (4, 40, 1028, "fp32"), (8, 600, 132, "fp32"), (8, 400, 8192, "bf16"), (4, 500, 5000, "fp16"), (8, 320, 4096, "fp32"),
    (6, 200, 8200, "bf16"), (16, 170, 4224, "fp32"), (1, 400, 16392, "bf16"),
    # the pipeline kernel with four and eight vectors per thread, and with several teams whose last tile is not full
    (4, 391, 16384, "fp16"), (3, 401, 10000, "bf16"), (2, 303, 8192, "fp32"), (2, 231, 16384, "fp32"), (1, 301, 32768, "bf16"),
    (1, 4099, 1024, "bf16"), (3, 1001, 2056, "fp16"), (2, 2601, 1000, "fp32"),
    # three vectors per thread
    (8, 411, 6144, "bf16"), (4, 391, 9352, "fp16"), (16, 803, 2192, "bf16"), (2, 401, 4728, "fp32"),
    # five to eight, rows of more than 32 KB
    (1, 201, 9000, "fp32"), (8, 111, 18000, "bf16"), (2, 167, 11004, "fp32"), (6, 83, 24008, "fp16"), (4, 161, 13004, "fp32"),
    (1, 333, 27000, "bf16"), (4, 171, 16384, "fp32"), (16, 160, 30008, "bf16"),
]


@pytest.mark.parametrize("W,M,N,dtype", CASES)
@pytest.mark.parametrize("kind", KINDS)
def test_matches_definition(car, W, M, N, dtype, kind):
    xs, res, w = make(W, M, N, dtype, seed=W * 1000 + M + N)
    h, y = normalised(xs, res, w, 1e-6)
    t, out = TORCH_DTYPE[dtype], Guarded()
    ro, no, ar = (out.empty((M, N), t) for _ in range(3))
    q = out.empty((M, N), torch.float8_e4m3fn)
    with car.Car(W, M, N, dtype) as c:
        shape = c.quant_scales_shape(kind)
        s = out.empty(shape, torch.uint8 if kind == "mx32" else torch.float32)
        if kind == "static":
            s.fill_(0.01)
        for extra in (False, True):
            q.view(torch.uint8).fill_(0x33)
            c.reduce_residual_rmsnorm_quant(xs, res, w, 1e-6, kind, ro, q, s, *((no, ar) if extra else ()))
            c.sync()
            sv = torch.full_like(y, float(s.double())) if kind == "static" else check_scales(kind, s, y)
            check_codes(q, y / sv, "q")
            assert torch.equal(ro, h.to(t))
    out.check()
    assert torch.equal(ar, rank_sum(xs).to(t))
    assert_within(no, y, (half(dtype) + DELTA) * y.abs() + TINY[dtype], "norm_out")


def test_residual_in_place_and_input_as_ar(car):
    W, M, N = 4, 37, 1032
    xs, res, w = make(W, M, N, "bf16", seed=5)
    h, y = normalised(xs, res, w, 1e-5)
    want_ar = rank_sum(xs).bfloat16()
    q = torch.empty(M, N, dtype=torch.float8_e4m3fn, device=DEV)
    s = torch.empty(M, 1, device=DEV)
    with car.Car(W, M, N, "bf16") as c:
        c.reduce_residual_rmsnorm_quant(xs, res, w, 1e-5, "row", res, q, s, ar_out=xs[2])
        c.sync()
    assert torch.equal(res, h.bfloat16()) and torch.equal(xs[2], want_ar)
    check_codes(q, y / check_scales("row", s, y), "q")


@pytest.mark.parametrize("W,M,N", [(2, 6, 512), (8, 3, 8192), (4, 400, 8192)])
@pytest.mark.parametrize("kind", KINDS)
def test_zero_rows_and_values_that_are_not_finite(car, W, M, N, kind):
    xs, res, w = make(W, M, N, "bf16", seed=11)
    for x in xs:
        x[0] = 0
        x[2] = 0
    res[0] = 0                    # a row of zeros: codes 0, the smallest scale
    res[1, 40] = float("nan")     # the statistic, so the whole row
    res[2] = 0
    res[2, 300] = 1.0e-30         # tiny, not zero: rms is 1 / sqrt(eps)
    w[100] = float("inf")         # one column of every row
    q = torch.empty(M, N, dtype=torch.float8_e4m3fn, device=DEV)
    with car.Car(W, M, N, "bf16") as c:
        s = torch.empty(c.quant_scales_shape(kind), device=DEV, dtype=torch.uint8 if kind == "mx32" else torch.float32)
        if kind == "static":
            s.fill_(2.0)
        ro = torch.empty_like(res)
        c.reduce_residual_rmsnorm_quant(xs, res, w, 1e-6, kind, ro, q, s)
        c.sync()
    v = q.float()
    assert v[1].isnan().all()
    if kind == "static":
        assert (v[0, :100] == 0).all() and v[0, 100].isnan()      # 0 * inf
        assert v[2, 300] == 0 and v[2, 100].isnan()
        fine = torch.arange(N, device=DEV) != 100
        # only row 1 and column 100 (saturated where the row is not 0 there)
        assert v[0][fine].isfinite().all() and v[2][fine].isfinite().all()
        return
    width = WIDTH.get(kind, N)
    sv = torch.where(s == 255, torch.nan, scale_values(s)) if kind == "mx32" else s
    sv = spread(sv, width, N)
    hit = 100 // width
    group = torch.arange(N, device=DEV) // width == hit
    for row in (0, 2):
        assert sv[row][group].isnan().all() and v[row][group].isnan().all()
        assert (v[row][~group] if kind == "row" else v[row][~group].nan_to_num(7.0)).isfinite().all()
    if kind != "row":
        assert (sv[0][~group] == 2.0**-126).all() and (v[0][~group] == 0).all()
        assert v[2, 300].item() == pytest.approx(res[2, 300].item() * 1e3 * w[300].item() / sv[2, 300].item(), rel=2.0**-4)


def test_row_of_zeros_alone_gets_the_smallest_scale(car):
    z = torch.zeros(3, 256, device=DEV, dtype=torch.float16)
    q = torch.empty(3, 256, dtype=torch.float8_e4m3fn, device=DEV)
    s = torch.empty(3, 1, device=DEV)
    with car.Car(1, 3, 256, "fp16") as c:
        c.reduce_residual_rmsnorm_quant([z], z, torch.ones(256, device=DEV).half(), 1e-6, "row", torch.empty_like(z), q, s)
        c.sync()
    assert (s == 2.0**-126).all() and (q.float() == 0).all()


def test_static_scale_saturates(car):
    M, N = 4, 512
    xs, res, w = make(2, M, N, "bf16", seed=8)
    _, y = normalised(xs, res, w, 1e-6)
    q = torch.empty(M, N, dtype=torch.float8_e4m3fn, device=DEV)
    s = torch.full((1,), 1e-4, device=DEV)
    with car.Car(2, M, N, "bf16") as c:
        c.reduce_residual_rmsnorm_quant(xs, res, w, 1e-6, "static", torch.empty_like(res), q, s)
        c.sync()
    big = (y.abs() > 0.05)
    assert (q.float().abs()[big] == 448).all() and s.item() == torch.tensor(1e-4).item()


@pytest.mark.parametrize("amax,k", [(448.0, 127), (448.0 * 2**-7, 120), (449.0, 128), (1.0, 119), (224.5, 127)])
def test_mx32_exponent_at_its_borders(car, amax, k):
    """One vector of ones normalises to itself (eps 0), so amax is the weight's largest value."""
    N = 64
    h = torch.ones(1, N, device=DEV)
    w = torch.full((N,), amax / 4, device=DEV)
    w[3] = amax
    w[40] = -amax if amax != 1.0 else -1.0
    q = torch.empty(1, N, dtype=torch.float8_e4m3fn, device=DEV)
    s = torch.empty(1, 2, dtype=torch.uint8, device=DEV)
    with car.Car(1, 1, N, "fp32") as c:
        c.reduce_residual_rmsnorm_quant([torch.zeros_like(h)], h, w, 0.0, "mx32", torch.empty_like(h), q, s)
        c.sync()
    assert s.tolist() == [[k, k]]
    assert q.float()[0, 3].item() * math.ldexp(1, k - 127) == pytest.approx(amax, rel=2.0**-4)


@pytest.mark.parametrize("W,M,N", [(8, 1, 8192), (2, 200, 4104), (4, 400, 8192)])
def test_captured_and_replayed_on_another_stream(car, W, M, N):
    xs, res, w = make(W, M, N, "bf16", seed=21)
    q = torch.empty(M, N, dtype=torch.float8_e4m3fn, device=DEV)
    ro = torch.empty_like(res)
    with car.Car(W, M, N, "bf16") as c:
        s = torch.empty(c.quant_scales_shape("group128"), device=DEV)
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            c.reduce_residual_rmsnorm_quant(xs, res, w, 1e-6, "group128", ro, q, s)
        for seed in (22, 23):
            nx, nr, nw = make(W, M, N, "bf16", seed=seed)
            for a, b in zip(xs + [res, w], nx + [nr, nw]):
                a.copy_(b)
            graph.replay()
            c.sync()
            h, y = normalised(xs, res, w, 1e-6)
            assert torch.equal(ro, h.bfloat16())
            check_codes(q, y / check_scales("group128", s, y), "q")
        del graph


def test_refusals(car):
    W, M, N = 2, 4, 64
    xs, res, w = make(W, M, N, "bf16", seed=1)
    q = torch.empty(M, N, dtype=torch.uint8, device=DEV)
    s = torch.empty(M, 2, device=DEV)
    with car.Car(W, M, N, "bf16") as c:
        P = lambda t: t.data_ptr()  # noqa: E731
        ok = dict(h=c.h, inputs=[P(x) for x in xs], residual=P(res), weight=P(w), eps=1e-6, kind=0, residual_out=P(res),
                  q_out=P(q), scales=P(s), norm_out=None, ar_out=None, stream=0)
        call = lambda **k: car.car_reduce_residual_rmsnorm_quant(**{**ok, **k})  # noqa: E731
        for k in (dict(kind=4), dict(kind=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(q_out=None), dict(scales=None),
                  dict(residual=None), dict(weight=None), dict(inputs=None), dict(residual_out=None)):
            assert call(**k) == car.CAR_ERR_ARG, k
        for k in (dict(q_out=P(q) + 4), dict(scales=P(s) + 2), dict(norm_out=P(q) + 2), dict(ar_out=P(q) + 8)):
            assert call(**k) == car.CAR_ERR_ALIGN, k
        assert car.car_quant_scale_bytes(c.h, 9) == 0
        with pytest.raises(ValueError):
            c.reduce_residual_rmsnorm_quant(xs, res, w, 1e-6, "block", res, q, s)
        with pytest.raises(ValueError):
            c.reduce_residual_rmsnorm_quant(xs, res, w, 1e-6, "row", res, q[:2], s)
        with pytest.raises(ValueError):
            c.reduce_residual_rmsnorm_quant(xs, res, w, 1e-6, "group128", res, q, s[0, :1])
    with car.Car(1, 1, 40000, "bf16") as c:
        x = torch.zeros(1, 40000, device=DEV).bfloat16()
        with pytest.raises(car.CarError) as e:
            c.reduce_residual_rmsnorm_quant([x], x, x[0], 1e-6, "row", x, torch.empty(1, 40000, dtype=torch.uint8, device=DEV),
                                            torch.empty(1, 1, device=DEV))
        assert e.value.status == car.CAR_ERR_SIZE
