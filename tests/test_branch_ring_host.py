"""The ring of the branch pipelines has room whatever a call's parts are: for every row length, rank count, number of teams and
set of slices that the kernels' shapes allow, a ring of at least six slices fits beside the weights, so that which kernel runs
depends on the handle alone.  Calls the library's own rule; no test here launches a kernel."""
import ctypes

import pytest

BUDGET = 224 * 1024


class RingPlan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("rows", "row_bytes", "vec_per_row", "cluster", "chunk", "ranks", "held", "group",
                                            "tile_stages", "stages", "teams", "producers", "team_threads")] + [
        ("gate_span", ctypes.c_uint32)]


@pytest.fixture(scope="module")
def fit():
    import __graft_entry__

    __graft_entry__.build()
    import rank_sum_reduce_gb300 as car

    f = ctypes.CDLL(car.LIB_PATH)["_ZN3car15branch_ring_fitEiPNS_8RingPlanE"]
    f.argtypes, f.restype = [ctypes.c_int, ctypes.POINTER(RingPlan)], ctypes.c_bool
    return f


def check(fit, beside, ranks, held, teams, chunk):
    p = RingPlan(ranks=ranks, held=held, teams=teams, chunk=chunk)
    what = (beside, ranks, held, teams, chunk)
    assert fit(BUDGET - beside, ctypes.byref(p)) and p.stages >= 2 and p.stages * p.group >= 6, what
    assert p.stages * p.group * teams * chunk * 16 + beside <= BUDGET, what
    # the stages of a tile: one of all slices, or the ranks' and one of those that a row holds to its end
    assert p.tile_stages == (1 if p.group == ranks + held else -(-ranks // p.group) + 1), what


def shapes(last_whole, last_pair, vpts):
    """(vectors of a row in one CTA, teams)."""
    seen = set()
    for V in range(1, 4097):
        cluster = 4 if V > last_pair else 2 if V > last_whole else 1
        chunk = -(-V // cluster)
        for vpt in vpts:
            threads = -(-(-(-chunk // vpt)) // 32) * 32
            if threads <= 512:
                seen |= {(chunk, t) for t in (range(1, 512 // threads + 1) if cluster == 1 else (1,))}
    # the fewest and the most vectors of every (teams, 16 vectors) stand for those between
    return sorted(s for s in seen if s[0] % 16 in (0, 1) or s[0] < 64)


def test_forward(fit):
    for chunk, teams in shapes(1536, 2048, (2, 3)):
        for ranks in range(1, 17):
            for rows in (1, 2, 3):            # weights beside the ring
                for held in (1, 2):
                    check(fit, rows * chunk * 16, ranks, held, teams, chunk)


def test_backward(fit):
    for chunk, teams in shapes(1024, 2048, (2,)):
        for ranks in range(1, 17):
            for held in (1, 2, 3, 4):
                for wide in (1, 2):           # a weight's bytes by a vector's: 16-bit types in fp32
                    for factor in (0, 1):
                        check(fit, (1 + factor + (teams if teams > 1 else 0)) * wide * chunk * 16, ranks, held, teams, chunk)
