"""Few rows of experts that do not fall alike, in the products that take them straight to registers: as many blocks as there
can be passes of eight rows, however the rows fall. No GPU."""
from __future__ import annotations

import ctypes
import random

import pytest

from test_fp8_plan import ROOM, lib  # noqa: F401  (the library is a fixture)


def falls(R, E):
    """Ways in which R rows fall among E experts."""
    rng = random.Random(R * 1000 + E)
    yield [R] + [0] * (E - 1)
    live = min(R, E)
    yield [R - live + 1] + [1] * (live - 1)
    yield [R // live + (i < R % live) for i in range(live)]
    nines = min(live, R // 9)
    if nines:
        yield [9] * (nines - 1) + [R - 9 * (nines - 1)]
    for _ in range(200):
        cuts = sorted(rng.randint(0, R) if rng.random() < 0.7 else 0 for _ in range(E - 1))
        yield [b - a for a, b in zip([0] + cuts, cuts + [R])]


@pytest.mark.parametrize("R,E", [(2, 2), (9, 2), (17, 3), (64, 8), (512, 256), (512, 2), (511, 512), (100, 7), (512, 30)])
def test_every_pass_has_a_block(lib, R, E):  # noqa: F811
    blocks = lib.plan_most_tiles(ctypes.c_int64(R), E, 8)
    most = 0
    for counts in falls(R, E):
        assert sum(counts) == R and len(counts) <= E
        passes = sum(-(-c // 8) for c in counts)
        assert passes <= blocks
        most = max(most, passes)
    assert most == blocks  # and none that no rows could need


def test_the_skewed_cases_go_straight_to_registers(lib):  # noqa: F811
    """Those that tests/test_fp8_skew_gpu.py runs."""
    room = (ctypes.c_int * 4)(*ROOM)
    experts = (31, 32, 33, 255, 256, 257, 300, 511, 512)
    for R, E, N, K in (*((r, e, 130, 144) for e in experts for r in (e // 2 + 2, 400)), (512, 256, 1383, 1152), (512, 256, 520, 400), (300, 40, 700, 528), (64, 256, 2565, 272)):
        assert lib.plan_small(ctypes.c_int64(R), E, ctypes.c_int64(N), K, room)
