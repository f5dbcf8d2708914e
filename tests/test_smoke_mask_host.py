"""The generator that smoke() compares the dropout's mask with: the published vectors of Philox4x32-10, the tests' own
generator, and mistakes that a mask's rate alone would not show.  No test here launches a kernel."""
import inspect

import numpy as np
import pytest


def bits(counter, key):
    """Of a whole counter and key, [4] and [2] words."""
    import __graft_entry__ as g

    return g._dropout_bits(key[0] | key[1] << 32, counter[2] | counter[3] << 32, counter[0] | counter[1] << 32)


@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_published_vectors(counter, key, want):
    assert bits(counter, key) == [half for word in want for half in (word & 0xFFFF, word >> 16)]


def test_the_tests_generator():
    from branch_checks import philox

    words = np.random.default_rng(3).integers(0, 2**32, (50, 6), dtype=np.uint64)
    for row in words:
        w = philox(row[None, :4], row[4:])[0].tolist()
        assert bits([int(v) for v in row[:4]], [int(v) for v in row[4:]]) == [h for word in w for h in (word & 0xFFFF, word >> 16)]


@pytest.mark.parametrize("right,wrong", [("range(10)", "range(9)"), ("0xD2511F53", "0xD2511F55"), ("0x9E3779B9", "0x9E3779B1"),
                                         ("(word & 0xFFFF, word >> 16)", "(word >> 16, word & 0xFFFF)"),
                                         ("offset >> 32", "0"), ("seed >> 32", "0")])
def test_a_mistake_changes_the_masks_that_smoke_looks_at(right, wrong):
    """Planted here, in the definition: a kernel with the same mistake would differ from the right one as much."""
    import __graft_entry__ as g

    text = inspect.getsource(g._dropout_bits)
    assert right in text
    scope = {}
    exec(text.replace(right, wrong), scope)
    seed, offset = 2**63 + 7, 2**40 + 11
    for M, N in ((6, 2056), (700, 1024), (160, 16384)):
        masks = [[[b >= 16384 for b in f(seed, offset, c)] for c in (0, 1, M * N // 16, M * N // 8 - 1)]
                 for f in (g._dropout_bits, scope["_dropout_bits"])]
        assert masks[0] != masks[1]
