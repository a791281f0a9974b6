"""Outputs and workspaces of the FP8 calls and of those around the experts come from the pool of the stream
that writes them: no GPU (the allocator, the streams and the library are stood in for)."""
from __future__ import annotations

import pytest
import torch

import sandwich_norm_residual_gb300 as snr
from test_output_streams import E, H, IDX, MAIN, SIDE, TW, W, X, D, T, made  # noqa: F401  (made is a fixture)

A8, S8 = torch.zeros((T, D), dtype=torch.float8_e4m3fn), torch.zeros((T, 1))
W8, SW = torch.zeros((2, T, D), dtype=torch.float8_e4m3fn), torch.zeros((2, 1, 1))
OFF, SLOTS = torch.zeros(3, dtype=torch.int32), torch.zeros((T, 8), dtype=torch.int32)

CALLS = {  # tensors made, call
    "boundary_fused_fp8": (2, lambda **k: snr.boundary_fused_fp8(H, X, W, W, 2, **k)),
    "moe_combine_boundary_fp8": (2, lambda **k: snr.moe_combine_boundary_fp8(H, E, TW, W, W, 2, **k)),
    "matmul_fp8": (1, lambda **k: snr.matmul_fp8(A8, S8, W8[0], SW[0], **k)),
    "matmul_fp8_experts": (1, lambda **k: snr.matmul_fp8_experts(A8, S8, OFF, W8, SW, **k)),
    "swiglu_fp8": (2, lambda **k: snr.swiglu_fp8(X, OFF, **k)),
    "moe_sort": (3, lambda **k: snr.moe_sort(IDX, 2, **k)),
    "moe_gather": (1, lambda **k: snr.moe_gather(H, SLOTS, **k)),
    "moe_gather_scales": (2, lambda **k: snr.moe_gather(A8, SLOTS, S8, **k)),
    "moe_gather_backward": (1, lambda **k: snr.moe_gather_backward(H, SLOTS, **k)),
    "moe_combine": (1, lambda **k: snr.moe_combine(H, SLOTS, TW, **k)),
    "moe_combine_backward": (2, lambda **k: snr.moe_combine_backward(X, H, SLOTS, TW, **k)),
}


@pytest.fixture(autouse=True)
def fresh_workspaces():
    snr._sort_workspace.cache_clear()
    yield
    snr._sort_workspace.cache_clear()


@pytest.mark.parametrize("name", CALLS)
def test_tensors_come_from_the_stream_that_writes_them(made, name):  # noqa: F811
    n, call = CALLS[name]
    current, got, entered = made
    call(stream=SIDE)
    assert got == [SIDE] * n
    assert current == [MAIN] and entered == [SIDE]  # entered once a call
    got.clear()
    call()
    assert got == [MAIN] * n


@pytest.mark.parametrize("name", CALLS)
def test_the_current_stream_is_not_entered_again(made, name):  # noqa: F811
    n, call = CALLS[name]
    current, got, entered = made
    call(stream=MAIN)
    assert got == [MAIN] * n and entered == []
