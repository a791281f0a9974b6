"""How the 8-bit integer product is divided, on the host (csrc/matmul_int8_plan.h, compiled by g++):
the largest sizes, every SM count, workspaces. No GPU."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest

from sandwich_norm_residual_gb300 import _lib, build

HERE = os.path.dirname(os.path.abspath(__file__))
TOP = 2 ** 31 - 1
TILES = {1: (16, 1), 2: (32, 1), 3: (64, 1), 4: (128, 1), 5: (256, 2)}  # tokens, CTAs of a tile
FIELDS = ("m_tiles", "steps", "tiles", "waves", "workers", "sharers", "split", "bytes")


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    so = tmp_path_factory.mktemp("plan") / "libplan.so"
    subprocess.run(["g++", "-std=c++20", "-O1", "-fPIC", "-shared", f"-I{build.CSRC}",
                    os.path.join(HERE, "matmul_int8_plan.cpp"), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    lib.plan_choose.argtypes = lib.plan_workspace.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int]
    lib.plan_workspace.restype = ctypes.c_int64
    return lib


def fields(lib, name, shape, M, N, K, sms):
    out = (ctypes.c_int64 * 8)()
    getattr(lib, name)(ctypes.c_int(shape), ctypes.c_int64(M), ctypes.c_int64(N), ctypes.c_int(K), ctypes.c_int(sms),
                       out)
    return dict(zip(FIELDS, out))


@pytest.mark.parametrize("N", [TOP, TOP - 7, 2 ** 31 - 128, 2 ** 31 - 256, 2 ** 31 - 300])
def test_channels_up_to_the_last_31_bit_number(lib, N):
    for shape, (nt, cg) in TILES.items():
        for K in (16, 65536):
            q = fields(lib, "plan_fields", shape, 9, N, K, 152)
            assert q["tiles"] == -(-N // (128 * cg)) and q["steps"] == -(-K // 128)
            last = (q["tiles"] - 1) * 128 * cg + 128 * (cg - 1)  # the last CTA's first channel
            assert last < 2 ** 31
            for n0 in (0, 128, last - 128, last):
                assert lib.plan_whole_channels(N, n0) == (n0 + 128 <= N)
        assert lib.plan_workspace(9, N, 16) >= 0


def test_the_library_sizes_workspaces_alike(lib):
    build.build()
    ws = _lib.load().beam_matmul_int8_workspace
    for M, N, K in ((1, 6144, 5120), (9, TOP - 7, 16), (16, TOP, 65536), (64, 5120, 20480), (517, 2565, 2576),
                    (700, 5120, 2560), (1030, 5110, 2064)):
        assert ws(M, N, K) == lib.plan_workspace(M, N, K)


def test_every_step_of_every_tile_is_taken_once(lib):
    for shape, (nt, cg) in TILES.items():
        for M, N, K in ((9, 70, 16), (64, 5120, 20480), (517, 2565, 2576), (1030, 5110, 2064), (300, 20480, 5120)):
            q = fields(lib, "plan_fields", shape, M, N, K, 152)
            tiles, steps = q["tiles"], q["steps"]
            assert tiles == -(-M // nt) * -(-N // (128 * cg))
            whole = min(tiles, q["waves"] * q["workers"])
            assert q["split"] in (0, (tiles - whole) * steps)
            if q["split"] == 0:
                assert whole == tiles
            else:
                cuts = [q["split"] * c // q["sharers"] for c in range(q["sharers"] + 1)]
                assert all(a < b for a, b in zip(cuts, cuts[1:])) and cuts[-1] == q["split"]
                assert q["bytes"] == q["sharers"] * cg * 2 * nt * 128 * 4


def test_a_launch_on_fewer_sms_needs_no_more_than_the_workspace_that_was_asked_for(lib):
    """152 tiles are one wave of 152 SMs and need none; 148 SMs would share the last four."""
    shapes = [(100, 152 * 128, 5120), (64, 5120, 20480), (300, 20480, 5120), (1030, 5110, 2064), (9, 70, 16),
              (2048, 76 * 256, 20480)]
    seen = 0
    for M, N, K in shapes:
        shape, need = lib.plan_choose(M, N, K), lib.plan_workspace(M, N, K)
        for sms in range(2, 200):
            raw = fields(lib, "plan_fields", shape, M, N, K, sms)
            q = fields(lib, "launch_fields", shape, M, N, K, sms)
            assert q["bytes"] <= need
            seen += raw["bytes"] > need and sms < 152
            if q["split"] == 0:  # whole tiles then cover everything
                assert q["waves"] * q["workers"] >= q["tiles"]
            else:
                assert q["split"] == (q["tiles"] - q["waves"] * q["workers"]) * q["steps"]
            assert q["workers"] <= 152
    assert fields(lib, "plan_fields", lib.plan_choose(100, 152 * 128, 5120), 100, 152 * 128, 5120, 148)["bytes"] > 0
    assert lib.plan_workspace(100, 152 * 128, 5120) == 0 and seen
