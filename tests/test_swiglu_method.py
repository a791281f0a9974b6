"""Steps of the experts' activation in FP32 with the worst base-2 exponential and reciprocal that the hardware's
bounds allow: y within (8 + 2 |g|) 2^-24 at every BF16 gate whose e^-g is an FP32 number. No GPU."""
from __future__ import annotations

import numpy as np
import pytest

F = np.float32
LOG2E = F(1.4426950408889634)
DOWN = F(2.0 ** -32)


def flushed(v):
    """To FP32, results below 2^-126 to 0."""
    v = v.astype(F)
    return np.where(np.abs(v) < F(2.0 ** -126), F(0), v)


@pytest.mark.parametrize("ex2", [-1, 0, 1])
@pytest.mark.parametrize("rcp", [-1, 0, 1])
@pytest.mark.parametrize("u", [1.0, -2.0 ** 60, 3.3e38])
def test_every_gate(ex2, rcp, u):
    """2^x off by 2^-22 and 1 / d by 2^-23, up or down; silu and y round to multiples of 2^-149."""
    g = (np.arange(65536, dtype=np.uint32) << 16).view(F)
    g = g[np.isfinite(g) & (g > -88.72)]
    g64 = g.astype(np.float64)
    with np.errstate(over="ignore", under="ignore"):
        t = flushed(np.exp2((g * -LOG2E).astype(np.float64)) * (1 + ex2 * 2.0 ** -22))
        assert np.isfinite(t).all()
        # exact in 64 bits before its one rounding
        d = (t.astype(np.float64) * float(DOWN) + float(DOWN)).astype(F)
        r = flushed(1 / d.astype(np.float64) * (1 + rcp * 2.0 ** -23))
        assert (r > 0).all()
        silu = g * (r * DOWN)
        exact = g64 / (1 + np.exp(-g64))
        y = silu * F(u)
        want = exact * np.float64(F(u))
    fits = np.abs(want) * (1 + 2.0 ** -16) < np.finfo(F).max
    tol = (8 + 2 * np.abs(g64)) * 2.0 ** -24 * np.abs(want) + 2.0 ** -149 * (1 + abs(u))
    assert (np.abs(y.astype(np.float64) - want) <= tol)[fits].all()
    assert np.isinf(y[np.abs(want) * (1 - 2.0 ** -16) > np.finfo(F).max]).all()


def test_gates_whose_exponential_overflows():
    x = np.array([-88.5, -89.0], F) * -LOG2E
    assert (x < 128).tolist() == [True, False]
