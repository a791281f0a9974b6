"""Sizes and numbers past 32 bits, which the C ABI takes as int, are refused and not cut: no GPU
(tensors without memory, on the meta device)."""
from __future__ import annotations

import pytest
import torch

import sandwich_norm_residual_gb300 as snr
from sandwich_norm_residual_gb300 import _lib

BIG = 2 ** 32  # cut to 32 bits, BIG + n is n


class NoLibrary:
    def __getattr__(self, name):
        if name.endswith("_workspace"):
            return lambda *a: 0


        def reached(*args):
            raise AssertionError(f"{name} was called")
        return reached


@pytest.fixture(autouse=True)
def bound(monkeypatch):
    monkeypatch.setattr(snr, "_on_current_device", lambda **k: None)
    monkeypatch.setattr(snr, "_raw_stream", lambda *a: None)
    monkeypatch.setattr(snr, "_stream_ptr", lambda *a: None)
    monkeypatch.setattr(_lib, "_lib", NoLibrary())
    for f in (snr._matmul_workspace, snr._balance_workspace):
        f.cache_clear()
    yield
    for f in (snr._matmul_workspace, snr._balance_workspace):
        f.cache_clear()


def meta(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")


def bf(*shape):
    return meta(*shape, dtype=torch.bfloat16)


def i8(*shape):
    return meta(*shape, dtype=torch.int8)


def i32(*shape):
    return meta(*shape, dtype=torch.int32)


D = BIG + 64
CASES = {
    "boundary": lambda: snr.boundary_fused(bf(2, D), bf(2, D), bf(D), bf(D), 2),
    "boundary n": lambda: snr.boundary_fused(bf(2, 64), bf(2, 64), bf(64), bf(64), BIG + 2),
    "moe": lambda: snr.moe_combine_boundary(bf(2, D), bf(2, 8, D), meta(2, 8), bf(D), bf(D), 2),
    "moe scaled": lambda: snr.moe_combine_boundary(bf(2, D), bf(2, 8, D), meta(2, 8), bf(D), bf(D), 2,
                                                   route_scale=1.5),
    "nvfp4": lambda: snr.boundary_fused_nvfp4(bf(2, D), bf(2, D), bf(D), bf(D), 2, 1e-6, 1.0),
    "moe nvfp4": lambda: snr.moe_combine_boundary_nvfp4(bf(2, D), bf(2, 8, D), meta(2, 8), bf(D), bf(D), 2, 1e-6, 1.0),
    "int8": lambda: snr.boundary_fused_int8(bf(2, D), bf(2, D), bf(D), bf(D), 2),
    "moe int8": lambda: snr.moe_combine_boundary_int8(bf(2, D), bf(2, 8, D), meta(2, 8), bf(D), bf(D), 2),
    "product K": lambda: snr.matmul_int8(i8(3, D), meta(3), i8(5, D), meta(5)),
    "product N": lambda: snr.matmul_int8(i8(3, 64), meta(3), i8(BIG + 5, 64), meta(BIG + 5)),
    "route": lambda: snr.moe_route(meta(2, BIG + 256), meta(BIG + 256)),
    "route topk": lambda: snr.moe_route(meta(2, 256), meta(256), n_group=BIG + 8),
    "balance E": lambda: snr.moe_balance_loss(meta(2, BIG + 256), i32(2, 8), 1.0),
    "balance topk": lambda: snr.moe_balance_loss(meta(2, 256), i32(2, BIG + 8), 1.0),
    "balance backward E": lambda: snr.moe_balance_loss_backward(meta(1), meta(2, BIG + 256), i32(1, BIG + 256), 8, 1.0),
    "balance backward topk": lambda: snr.moe_balance_loss_backward(meta(1), meta(2, 256), i32(1, 256), BIG + 8, 1.0),
    "qk heads": lambda: snr.qk_norm(bf(2, BIG + 8, 128), bf(2, 8, 128), bf(128), bf(128), i32(2), mode="ssmax"),
}


@pytest.mark.parametrize("name", CASES)
def test_refused(name):
    with pytest.raises(ValueError, match="32-bit"):
        CASES[name]()
