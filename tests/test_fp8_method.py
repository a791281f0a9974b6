"""Steps of the FP8 quantiser in exact arithmetic: the division by 448 in three operations, the codes. No GPU."""
from __future__ import annotations

import numpy as np
import torch

C = np.float32(1) / np.float32(448)


def div448(a: np.ndarray) -> np.ndarray:
    """The kernels' steps; every fused multiply-add here is exact in 64 bits before its one rounding."""
    t = a * C
    r = (-t.astype(np.float64) * 448.0 + a.astype(np.float64)).astype(np.float32)
    exact = np.float64(r) * np.float64(C) + t.astype(np.float64)
    return exact.astype(np.float32)


def test_the_constant():
    assert C == np.float32(float.fromhex("0x1.24924ap-9"))


def test_division_by_448_rounds_correctly_for_every_significand():
    # scaling by a power of two changes nothing while no step leaves the normal numbers
    for e in (0, 1):
        bits = (np.arange(2 ** 23, dtype=np.uint32) | np.uint32((127 + e) << 23)).view(np.float32)
        assert np.array_equal(div448(bits), bits / np.float32(448))
    for e in (-100, -99, 0, 127):
        bits = (np.arange(0, 2 ** 23, 97, dtype=np.uint32) | np.uint32((127 + e) << 23)).view(np.float32)
        assert np.array_equal(div448(bits), bits / np.float32(448))


def test_the_second_product_is_exact_in_64_bits():
    """r c has at most 48 bits and lies within 2^24 of t's last place: 64 bits hold the sum to far below a
    rounding of it."""
    a = np.float32(1.9999999)
    t = a * C
    r = np.float64(a) - 448.0 * np.float64(t)
    assert abs(r * np.float64(C)) <= np.spacing(t) * 1.01


def test_codes_never_leave_448():
    """v times the inverse of the largest is at most 448 (1 + 2^-23), which rounds to 448."""
    top = torch.rand(100000, dtype=torch.float32) * 10 + 1e-3
    inv = torch.tensor(448.0) / top
    assert float((top * inv).max()) <= 448.0 * (1 + 2.0 ** -23)
    assert (torch.clamp(top * inv, max=448.0).to(torch.float8_e4m3fn).float() == 448).all()
