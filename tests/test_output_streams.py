"""Outputs and workspaces that a call makes come from the pool of the stream that writes them: no GPU.

The allocator, the streams and the library are stood in for; what is seen is which stream is current
when each tensor is made."""
from __future__ import annotations

import contextlib

import pytest
import torch

import sandwich_norm_residual_gb300 as snr
from sandwich_norm_residual_gb300 import _lib


class FakeStream:
    device_index = 0

    def __init__(self, handle):
        self.cuda_stream = handle


class FakeLibrary:
    def __getattr__(self, name):
        if name.endswith("_workspace"):
            return lambda *a: 64
        return lambda *a: 0


MAIN, SIDE = FakeStream(1), FakeStream(2)
bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
T, D = 4, 64
H, X, W, E, TW = bf(T, D), bf(T, D), bf(D), bf(T, 8, D), torch.zeros((T, 8))
A, S4 = torch.zeros((T, D), dtype=torch.int8), torch.zeros(T)
Z, IDX, C = torch.zeros((T, 256)), torch.zeros((T, 8), dtype=torch.int32), torch.zeros((1, 256), dtype=torch.int32)

CALLS = {  # tensors made, call
    "boundary_fused": (1, lambda **k: snr.boundary_fused(H, X, W, W, 2, **k)),
    "moe_combine_boundary": (1, lambda **k: snr.moe_combine_boundary(H, E, TW, W, W, 2, **k)),
    "boundary_fused_nvfp4": (2, lambda **k: snr.boundary_fused_nvfp4(H, X, W, W, 2, 1e-6, 1.0, **k)),
    "moe_combine_boundary_nvfp4": (2, lambda **k: snr.moe_combine_boundary_nvfp4(H, E, TW, W, W, 2, 1e-6, 1.0, **k)),
    "boundary_fused_int8": (2, lambda **k: snr.boundary_fused_int8(H, X, W, W, 2, **k)),
    "moe_combine_boundary_int8": (2, lambda **k: snr.moe_combine_boundary_int8(H, E, TW, W, W, 2, **k)),
    "matmul_int8": (2, lambda **k: snr.matmul_int8(A, S4, A, S4, **k)),
    "moe_route": (2, lambda **k: snr.moe_route(Z, Z[0], **k)),
    "moe_balance_loss": (3, lambda **k: snr.moe_balance_loss(Z, IDX, 1.0, **k)),
    "moe_balance_loss_backward": (1, lambda **k: snr.moe_balance_loss_backward(S4[:1], Z, C, 8, 1.0, **k)),
    "router_sigmoid": (1, lambda **k: snr.router_sigmoid(Z, **k)),
}


@pytest.fixture
def made(monkeypatch):
    """(the stream that is current, the streams that tensors were made under, the streams entered)"""
    current, made, entered = [MAIN], [], []

    @contextlib.contextmanager
    def stream(s):
        entered.append(s)
        current.append(s)
        yield
        current.pop()

    def recording(fn):
        def f(*args, **kw):
            kw.pop("device", None)
            made.append(current[-1])
            return fn(*args, **kw)
        return f

    for name in ("empty", "empty_like"):
        monkeypatch.setattr(torch, name, recording(getattr(torch, name)))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: current[-1].cuda_stream, raising=False)
    monkeypatch.setattr(snr, "_on_current_device", lambda **k: None)
    monkeypatch.setattr(snr, "_torch", torch)
    monkeypatch.setattr(_lib, "_lib", FakeLibrary())
    for f in (snr._matmul_workspace, snr._balance_workspace):
        f.cache_clear()
    yield current, made, entered
    for f in (snr._matmul_workspace, snr._balance_workspace):
        f.cache_clear()


@pytest.mark.parametrize("name", CALLS)
def test_tensors_come_from_the_stream_that_writes_them(made, name):
    n, call = CALLS[name]
    current, got, entered = made
    call(stream=SIDE)
    assert got == [SIDE] * n
    assert current == [MAIN] and entered == [SIDE]  # entered once a call
    got.clear()
    call()
    assert got == [MAIN] * n


@pytest.mark.parametrize("name", CALLS)
def test_the_current_stream_is_not_entered_again(made, name):
    n, call = CALLS[name]
    current, got, entered = made
    call(stream=MAIN)
    assert got == [MAIN] * n and entered == []


def test_a_bare_handle_is_a_stream(made, monkeypatch):
    """What the calls ask of a stream is its handle alone."""
    class Handle:
        cuda_stream = 2

    current, got, entered = made
    monkeypatch.setattr(torch.cuda, "ExternalStream", FakeStream)
    for name in ("boundary_fused", "moe_route", "matmul_int8"):
        CALLS[name][1](stream=Handle())
    assert [s.cuda_stream for s in entered] == [2, 2, 2] and all(s.cuda_stream == 2 for s in got)
