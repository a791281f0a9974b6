"""How the 8-bit floating-point product is divided (csrc/matmul_fp8_plan.h, compiled by g++): every row and
channel has one tile, clusters fit. No GPU."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest

from sandwich_norm_residual_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))
ROOM = (152, 76, 36, 15)  # clusters of 1, 2, 4 and 8 CTAs that a GB300 holds at a time


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    so = tmp_path_factory.mktemp("plan") / "libplan.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", f"-I{build.CSRC}",
                    os.path.join(HERE, "fp8_plan.cpp"), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    lib.plan_most_tiles.restype = ctypes.c_int64
    return lib


def plan(lib, R, E, N, K, room=ROOM):
    out = (ctypes.c_int64 * 4)()
    lib.plan_fields(ctypes.c_int64(R), E, ctypes.c_int64(N), K, (ctypes.c_int * 4)(*room), out)
    return dict(zip(("few", "width", "split", "clusters"), out))


def rows(lib, few, n):
    out = (ctypes.c_uint32 * 2)()
    lib.plan_rows(few, ctypes.c_uint32(n), out)
    return out[0], out[1]


@pytest.mark.parametrize("few,most,grain", [(1, 64, 16), (0, 128, 128)])
def test_rows_of_an_expert_have_a_tile_each(lib, few, most, grain):
    for n in list(range(1, 700)) + [2 ** 31 - 4097, 2 ** 31 - 4096]:
        tiles, each = rows(lib, few, n)
        assert tiles == -(-n // most) and each <= most and each % grain == 0
        assert (tiles - 1) * each < n <= tiles * each  # none is empty, none is left over
    assert rows(lib, few, 0)[0] == 0


@pytest.mark.parametrize("m,n", [(1, 1), (1, 40), (3, 7), (8, 5), (9, 5), (17, 20), (64, 3), (70, 1)])
def test_every_tile_has_one_number(lib, m, n):
    out, seen = (ctypes.c_uint32 * 2)(), set()
    for u in range(m * n):
        lib.plan_place(u, m, n, out)
        assert out[0] < m and out[1] < n
        seen.add((out[0], out[1]))
    assert len(seen) == m * n


@pytest.mark.parametrize("R,E", [(1, 1), (7, 8), (512, 256), (513, 4), (131072, 256), (100, 512)])
def test_bound_on_the_tiles_of_unknown_experts(lib, R, E):
    """However the rows fall, no more tiles than that."""
    import random
    rng = random.Random(R)
    for few, most in ((1, 64), (0, 128)):
        bound = lib.plan_most_tiles(ctypes.c_int64(R), E, most)
        for _ in range(50):
            weights = [rng.random() ** rng.choice([1, 8, 40]) for _ in range(E)]
            cuts = sorted(min(R, int(R * sum(weights[:i]) / sum(weights))) for i in range(1, E)) + [R]
            counts = [b - a for a, b in zip([0] + cuts, cuts)]
            assert sum(rows(lib, few, c)[0] for c in counts) <= bound
    assert lib.plan_most_tiles(ctypes.c_int64(R), 1, 64) == -(-R // 64)


@pytest.mark.parametrize("room", [ROOM, (152, 76, 36, 0), (148, 74, 0, 0), (4, 2, 1, 0), (1, 0, 0, 0)])
def test_plans_fit_the_device_and_take_every_step(lib, room):
    for R, E, N, K in [(1, 1, 128, 16), (2, 1, 6144, 5120), (64, 1, 5120, 20480), (517, 1, 2565, 2576), (65, 1, 1, 128),
                       (16384, 1, 20480, 5120), (1024, 1, 5120, 5120), (4096, 1, 5120, 5120), (17, 256, 5120, 5120),
                       (512, 256, 5120, 5120), (131072, 256, 5120, 2560), (40, 512, 130, 65536),
                       (2 ** 31 - 4096, 1, 16, 16)]:
        q = plan(lib, R, E, N, K, room)
        index = {1: 0, 2: 1, 4: 2, 8: 3}[q["split"]]
        assert 1 <= q["clusters"] <= room[index]
        assert q["split"] <= -(-K // 128)  # a share has a step at least
        assert q["width"] == 128 or (q["width"] == 256 and not q["few"])
        if R <= 32:
            assert q["few"]
        if not q["few"] and q["split"] > 1 and E == 1:
            # many tokens' shared tiles have one round at most
            tiles = -(-R // 128) * -(-N // q["width"])
            assert tiles % (q["clusters"] * q["split"]) <= q["clusters"]


def test_a_few_tokens_go_straight_to_registers(lib):
    room = (ctypes.c_int * 4)(*ROOM)
    small = lambda r, e, n, k: lib.plan_small(ctypes.c_int64(r), e, ctypes.c_int64(n), k, room)  # noqa: E731
    assert [small(r, 1, 6144, 5120) for r in (1, 8, 9, 16, 17, 64)] == [1, 1, 1, 1, 0, 0]
    assert [small(r, 1, 20480, 5120) for r in (1, 8, 9, 16)] == [1, 1, 0, 0]
    assert [small(8, 1, n, k) for n, k in ((640, 20480), (640, 20496), (4096, 65536))] == [1, 0, 1]
    assert [small(16, 1, n, k) for n, k in ((8192, 10240), (8193, 10240), (8192, 10256))] == [1, 0, 0]
    # experts: a token's choices, a few tokens' of many; not an expert's hundred rows, nor more rows than the kernel counts
    assert [small(*c) for c in ((8, 256, 5120, 5120), (55, 211, 1383, 1152), (300, 3, 1000, 640), (513, 256, 128, 128))] == [1, 1, 0, 0]
