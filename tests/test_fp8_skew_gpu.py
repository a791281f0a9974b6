"""Few rows of experts that do not fall alike, straight to registers: right, and not slower by the largest expert's rows."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import sandwich_norm_residual_gb300 as snr
from sandwich_norm_residual_gb300 import build
from test_matmul_fp8_gpu import check_experts, cuts, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    snr.library()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,N,K", [
    ([0] * 100 + [512] + [0] * 155, 1383, 1152), ([512] + [0] * 255, 520, 400), ([0] * 255 + [512], 520, 400),
    ([257] + [1] * 255, 520, 400), ([1] * 255 + [257], 520, 400), ([64] * 8 + [0] * 248, 1383, 1152),
    ([0] * 31 + [17, 9, 8, 24, 25] + [0] * 90 + [33] + [0] * 100 + [7, 65] + [0] * 27, 2565, 272),
    ([9] * 33 + [0] * 6 + [3], 700, 528), ([0, 8, 16, 0, 24, 7, 15, 23, 9, 17, 25, 1] + [0] * 27 + [155], 700, 528),
])
def test_rows_that_do_not_fall_alike(counts, N, K, dtype):
    check_experts(counts, N, K, dtype=dtype, seed=len(counts))


@pytest.mark.parametrize("E", [31, 32, 33, 255, 256, 257, 300, 511, 512])
def test_any_number_of_experts(E):
    """A lane looks at 1, 8 or 16 of them."""
    rng = np.random.default_rng(E)
    few = rng.integers(0, 2, E)
    few[-1] = 3
    check_experts(few.tolist(), 130, 144, seed=E)
    many = np.zeros(E, dtype=np.int64)
    many[rng.integers(0, E, 5)] += rng.integers(1, 60, 5)
    many[0], many[-1] = 9, 25
    check_experts(many.tolist(), 130, 144, R=400, before=7, seed=E)


def test_rows_before_and_behind_the_experts():
    counts = [0] * 50 + [100, 3] + [0] * 204
    check_experts(counts, 520, 400, R=512, before=41)


def time_of(ops, off, n=10):
    a, sa, w, sw = ops
    out = torch.empty(a.shape[0], w.shape[1], dtype=torch.bfloat16, device="cuda")
    snr.matmul_fp8_experts(a, sa, off, w, sw, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(n):
            snr.matmul_fp8_experts(a, sa, off, w, sw, out=out)
    best = float("inf")
    for _ in range(10):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        g.replay()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) / n)
    return best


def test_an_expert_with_all_rows_takes_no_longer_than_all_experts():
    """512 rows of one expert read one expert's channels, 512 rows of all read 256 times as many. An expert's rows taken
    eight after eight by the same blocks made the first 0.83 of the second; with blocks of their own it takes 0.39."""
    ops = inputs(512, 1383, 1152, 0, 256)
    alike = time_of(ops, cuts([2] * 256))
    skewed = time_of(ops, cuts([0] * 100 + [512] + [0] * 155))
    assert skewed <= 0.6 * alike, (skewed, alike)
