"""Shared by the tests of the operators next to the rank sum: inputs, guarded outputs, exact rank sums.

Tolerances.  DELTA bounds what the kernels' fp32 arithmetic can lose of a normalised value, relative: a sum of N
squares over at most 16 terms in a row and 13 levels of partial sums (29 roundings of 2^-24, halved by the root),
the division by N, the addition of eps, rsqrtf (2 units of 2^-23) and at most 6 products: 14.5 + 1 + 4 + 6 < 32
roundings of 2^-24 = 2^-19.  half(t) is half a step of an output type, relative; TINY its smallest half step.
"""
import torch

TORCH_DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DELTA = 2.0**-19
TINY = {"bf16": 2.0**-134, "fp16": 2.0**-25, "fp32": 2.0**-150}
DEV = "cuda:0"
PAD = 64  # guard elements on both sides of an output


def half(dtype):
    return torch.finfo(TORCH_DTYPE[dtype]).eps / 2


def gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def randn(g, shape, dtype, sigma=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * sigma).to(TORCH_DTYPE[dtype])


def rank_sum(xs):
    """The fp32 sum in rank order, bit for bit."""
    acc = xs[0].float()
    for x in xs[1:]:
        acc = acc + x.float()
    return acc


class Guarded:
    """Outputs between guard bands that must come back untouched."""

    def __init__(self):
        self.bands = []

    def empty(self, shape, dtype):
        n = 1
        for d in shape:
            n *= d
        size = torch.empty(0, dtype=dtype).element_size()
        raw = torch.full(((n + 2 * PAD) * size,), 0xA5, dtype=torch.uint8, device=DEV)
        self.bands.append((raw, PAD * size, (PAD + n) * size))
        return raw[PAD * size:(PAD + n) * size].view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        for raw, lo, hi in self.bands:
            assert (raw[:lo] == 0xA5).all() and (raw[hi:] == 0xA5).all(), "a guard band was written"


def assert_within(got, want, bound, what):
    got, want, bound = got.double(), want.double(), bound.double()
    bad = ~((got - want).abs() <= bound)
    if bad.any():
        at = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {at}: got {got[at].item()!r} "
                             f"want {want[at].item()!r} within {bound[at].item()!r}")
