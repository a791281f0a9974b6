"""Which kernels smoke()'s FP8 products take, by the library's own choice. No GPU."""
from __future__ import annotations

import ctypes

import __graft_entry__ as entry
from synth import DENSE_DECODE_T4
from test_fp8_plan import ROOM, lib, plan  # noqa: F401  (the library is a fixture)


def test_smoke_runs_both_kinds_of_tiles(lib):  # noqa: F811
    room, N, K = (ctypes.c_int * 4)(*ROOM), 256, DENSE_DECODE_T4.D
    assert all(m % DENSE_DECODE_T4.T == 0 for m in entry.TILED_PRODUCTS)
    assert not any(lib.plan_small(ctypes.c_int64(m), 1, ctypes.c_int64(N), K, room) for m in entry.TILED_PRODUCTS)
    assert [bool(plan(lib, m, 1, N, K)["few"]) for m in entry.TILED_PRODUCTS] == [True, False]
