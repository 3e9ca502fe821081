"""Tiles of groups, whole and half, on the host model of their pipeline and of its end."""
import os
import random
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from pair_protocol_model import Leak  # noqa: E402
from pair_tiles_model import Tiles  # noqa: E402

BOTH, EVEN = (True, True), (True, False)
WORK = {"one group": [(1, BOTH)], "one each": [(1, EVEN)] * 9, "fewer than the ring": [(2, BOTH), (0, BOTH), (1, EVEN)],
        "nothing": [(0, BOTH)] * 4, "nothing at the end": [(5, BOTH), (0, EVEN)], "nothing first": [(0, EVEN), (7, BOTH)],
        "mixed": [(4, BOTH), (0, BOTH), (4, EVEN), (1, BOTH), (9, EVEN), (0, BOTH), (3, BOTH)], "long": [(23, EVEN), (2, BOTH)],
        "no tile": []}
RINGS = [(6, 4), (5, 2), (2, 4), (3, 1)]  # the first is half tiles', the second whole ones'


def random_work(seed):
    rng = random.Random(seed)
    return [(rng.choice((0, 0, 1, 2, 3, 4, 8)), rng.choice((BOTH, EVEN))) for _ in range(rng.randint(0, 9))]


@pytest.mark.parametrize("stages,accs", RINGS)
@pytest.mark.parametrize("name", [*WORK, "random"])
def test_tiles_leave_nothing_behind(name, stages, accs):
    for seed in range(40):
        work = random_work(seed) if name == "random" else WORK[name]
        p = Tiles(seed, stages, accs, work)
        p.run()
        every = [(t, g) for t, (n, _) in enumerate(work) for g in range(n)]
        assert not p.slow and p.issued == [len(every)] * 2 and p.read == [every, every]


@pytest.mark.parametrize("stages,accs", RINGS)
@pytest.mark.parametrize("name", ["one each", "mixed", "long", "random"])
def test_tiles_whose_waits_expire_leave_nothing_behind(name, stages, accs):
    slow = 0
    for seed in range(300):
        work = random_work(seed) if name == "random" else WORK[name]
        p = Tiles(seed, stages, accs, work, expire=(0.001, 0.004, 0.016)[seed % 3])
        p.run()
        slow += p.slow
    assert slow > 50  # the model did go that way


def test_model_sees_an_issuer_that_waits_for_too_few_accumulators():
    # the end of two accumulators under a ring of four: arrivals of the last hand-overs reach a pair that has left
    leaks = 0
    for seed in range(150):
        try:
            Tiles(seed, 6, 4, WORK["mixed"], hand_back=2).run()
        except Leak:
            leaks += 1
    assert leaks > 10
