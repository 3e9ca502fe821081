"""The end of a CTA pair's pipeline on the host model of it: nothing in flight, nothing waited for in vain."""
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from pair_protocol_model import Leak, Pair  # noqa: E402

SIZES = [(3, 3, 4), (5, 4, 7), (6, 1, 2), (4, 9, 1), (2, 2, 9)]


@pytest.mark.parametrize("stages,tiles,kblocks", SIZES)
def test_pair_leaves_nothing_behind(stages, tiles, kblocks):
    for seed in range(60):
        p = Pair(seed, stages, tiles, kblocks)
        p.run()
        assert not p.slow and p.issued == [tiles * kblocks] * 2


@pytest.mark.parametrize("stages,tiles,kblocks", SIZES)
def test_pair_whose_waits_expire_leaves_nothing_behind(stages, tiles, kblocks):
    slow = uneven = 0
    for seed in range(600):
        p = Pair(seed, stages, tiles, kblocks, expire=(0.001, 0.004, 0.016)[seed % 3])
        p.run()
        slow += p.slow
        uneven += p.issued[0] != p.issued[1]
    # the model did go that way (no producer waits for a first pass of the ring)
    assert slow > 50 and (uneven > 5 or tiles * kblocks <= stages)


def test_model_sees_an_end_that_only_the_even_cta_waits_for():
    # nothing but expired waits shows it, and the signals to a CTA that has left show without any
    for expire in (0.0, 0.01):
        leaks = 0
        for seed in range(150):
            try:
                Pair(seed, rule="even", expire=expire).run()
            except Leak:
                leaks += 1
        assert leaks > 10
