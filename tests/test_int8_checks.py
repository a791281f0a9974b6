"""Refusals of the int8 calls, in the C ABI (before any CUDA call) and in the binding: no GPU."""
from __future__ import annotations

import ctypes

import pytest
import torch

import sandwich_norm_residual_gb300 as snr
from sandwich_norm_residual_gb300 import _lib, build

A = 0x7F0000000000  # fake device addresses: never dereferenced
D = 5120


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_boundary_int8_argument_errors(lib):
    H, X, PW, QW, Q, S = (A + (i << 32) for i in range(6))
    E, W = A + (6 << 32), A + (7 << 32)

    def dense(T=4, d=D, n=2, eps=1e-6, h=H, x=X, q=Q, s=S, opts=None):
        return lib.beam_boundary_fused_int8(None, h, x, PW, QW, n, eps, T, d, q, s, opts)

    def moe(T=4, d=D, h=H, e=E, w=W, rs=1.0, q=Q, s=S, opts=None):
        return lib.beam_moe_combine_boundary_int8(None, h, e, w, rs, PW, QW, 2, 1e-6, T, d, q, s, opts)

    for call in (dense, moe):
        assert call(d=12) == _lib.BEAM_ERR_SHAPE
        assert call(T=-1) == _lib.BEAM_ERR_SHAPE
        assert call(T=0, h=None, q=None, s=None) == _lib.BEAM_OK
        assert call(h=None) == _lib.BEAM_ERR_NULL
        assert call(q=None) == _lib.BEAM_ERR_NULL
        assert call(s=None) == _lib.BEAM_ERR_NULL
        assert call(q=Q + 8) == _lib.BEAM_ERR_ALIGN
        assert call(s=S + 4) == _lib.BEAM_ERR_ALIGN
        assert call(s=Q + 4 * D - 16) == _lib.BEAM_ERR_ALIAS  # scales over the codes
        assert call(q=H + 64) == _lib.BEAM_ERR_ALIAS          # codes inside h
        assert call(s=PW + 16) == _lib.BEAM_ERR_ALIAS         # scales inside a weight
        ring = _lib.LaunchOpts(stages=2)
        assert call(opts=ctypes.byref(ring)) == _lib.BEAM_ERR_ARG
        hook = _lib.LaunchOpts(flags=_lib.BEAM_OPT_TEST_WAIT_TIMEOUT)
        assert call(opts=ctypes.byref(hook)) == _lib.BEAM_ERR_ARG
        assert call() in (_lib.BEAM_ERR_CUDA, _lib.BEAM_ERR_DEVICE)
    assert dense(n=0) == _lib.BEAM_ERR_ARG
    assert dense(eps=float("nan")) == _lib.BEAM_ERR_ARG
    assert dense(q=X + 64) == _lib.BEAM_ERR_ALIAS
    assert dense(x=H + 2 * D) == _lib.BEAM_ERR_ALIAS          # x partly over h
    assert dense(x=H) in (_lib.BEAM_ERR_CUDA, _lib.BEAM_ERR_DEVICE)  # x may be h itself
    assert moe(rs=float("inf")) == _lib.BEAM_ERR_ARG
    assert moe(h=E + 4096) == _lib.BEAM_ERR_ALIAS
    assert moe(q=W) == _lib.BEAM_ERR_ALIAS


def bf(*shape, device="cpu"):
    return torch.zeros(shape, dtype=torch.bfloat16, device=device)


def test_binding_checks_the_int8_boundaries():
    T, d = 4, 64
    h, x, w = bf(T, d), bf(T, d), bf(d)
    with pytest.raises(ValueError, match="y_int8 must have shape"):
        snr.boundary_fused_int8(h, x, w, w, 2, y_int8=torch.zeros((T, d // 2), dtype=torch.int8))
    with pytest.raises(ValueError, match="y_scale must have shape"):
        snr.boundary_fused_int8(h, x, w, w, 2, y_scale=torch.zeros(T + 1))
    with pytest.raises(TypeError, match="y_int8 must be"):
        snr.boundary_fused_int8(h, x, w, w, 2, y_int8=torch.zeros((T, d), dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA tensors"):
        snr.boundary_fused_int8(h, x, w, w, 2)
    e, tw = bf(T, 8, d), torch.zeros((T, 8))
    with pytest.raises(ValueError, match="shape mismatch"):
        snr.moe_combine_boundary_int8(h, e[:3].contiguous(), tw, w, w, 2)
    with pytest.raises(ValueError, match="one device"):
        snr.moe_combine_boundary_int8(h, e, tw.to("meta"), w, w, 2)


def test_matmul_argument_errors(lib):
    AA, AS, W, WS, O, P = (A + (i << 33) for i in range(6))

    def mm(M=4, N=40, K=64, a=AA, sa=AS, w=W, sw=WS, ty=0, o=O, ws=P, nb=1 << 30, flags=0):
        return lib.beam_matmul_int8(None, a, sa, w, sw, M, N, K, ty, o, ws, nb, flags)

    assert mm(M=-1) == _lib.BEAM_ERR_SHAPE
    assert mm(M=1 << 31) == _lib.BEAM_ERR_SHAPE
    assert mm(N=-1) == _lib.BEAM_ERR_SHAPE
    for K in (0, 8, 24, -16, _lib.BEAM_MATMUL_MAX_K + 16):
        assert mm(K=K) == _lib.BEAM_ERR_SHAPE
    assert mm(ty=2) == _lib.BEAM_ERR_ARG
    assert mm(flags=_lib.BEAM_OPT_FORCE_EXACT_SUM) == _lib.BEAM_ERR_ARG
    assert mm(flags=_lib.BEAM_OPT_TEST_WAIT_TIMEOUT) == _lib.BEAM_ERR_ARG  # nothing waits for 8 tokens or fewer
    assert mm(M=0, a=None) == _lib.BEAM_OK
    assert mm(N=0, w=None) == _lib.BEAM_OK
    for name in ("a", "sa", "w", "sw", "o"):
        assert mm(**{name: None}) == _lib.BEAM_ERR_NULL
    assert mm(a=AA + 8) == _lib.BEAM_ERR_ALIGN
    assert mm(w=W + 4) == _lib.BEAM_ERR_ALIGN
    assert mm(sa=AS + 2) == _lib.BEAM_ERR_ALIGN
    assert mm(o=O + 1) == _lib.BEAM_ERR_ALIGN
    assert mm(o=O + 2, ty=1) == _lib.BEAM_ERR_ALIGN
    assert mm(o=AA + 64) == _lib.BEAM_ERR_ALIAS
    assert mm(o=W - 2) == _lib.BEAM_ERR_ALIAS
    assert mm(o=AS + 4) == _lib.BEAM_ERR_ALIAS
    assert mm(o=WS) == _lib.BEAM_ERR_ALIAS
    # workspaces, where the shape needs one
    need = lib.beam_matmul_int8_workspace
    assert need(4, 40, 64) == 0 and need(0, 40, 64) == 0 and need(4, 40, 24) == -1
    big = dict(M=64, N=5120, K=20480)
    assert need(64, 5120, 20480) > 0
    assert mm(nb=need(64, 5120, 20480) - 1, **big) == _lib.BEAM_ERR_ARG
    assert mm(ws=None, **big) == _lib.BEAM_ERR_NULL
    assert mm(ws=P + 4, **big) == _lib.BEAM_ERR_ALIGN
    assert mm(ws=W + 16, **big) == _lib.BEAM_ERR_ALIAS
    assert mm(ws=O + 64, **big) == _lib.BEAM_ERR_ALIAS
    assert mm(ws=None, nb=0) in (_lib.BEAM_ERR_CUDA, _lib.BEAM_ERR_DEVICE)
    for flags in (0, _lib.BEAM_OPT_PDL):
        assert mm(o=O + 2, flags=flags) in (_lib.BEAM_ERR_CUDA, _lib.BEAM_ERR_DEVICE)


def test_binding_checks_the_product():
    a, sa, w, sw = torch.zeros((4, 64), dtype=torch.int8), torch.zeros(4), torch.zeros((6, 64), dtype=torch.int8), \
        torch.zeros(6)
    for bad in ((a, sa, w[:, :32].contiguous(), sw), (a, sa[:3], w, sw), (a, sa, w, sw[:5])):
        with pytest.raises(ValueError, match="shape mismatch"):
            snr.matmul_int8(*bad)
    with pytest.raises(TypeError, match="a must be"):
        snr.matmul_int8(a.to(torch.uint8), sa, w, sw)
    with pytest.raises(ValueError, match="contiguous"):
        snr.matmul_int8(a, sa, torch.zeros((64, 6), dtype=torch.int8).t(), sw)
    with pytest.raises(TypeError, match="out_dtype"):
        snr.matmul_int8(a, sa, w, sw, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="out must have shape"):
        snr.matmul_int8(a, sa, w, sw, out=torch.zeros((4, 7), dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="out must be"):
        snr.matmul_int8(a, sa, w, sw, out_dtype=torch.float32, out=torch.zeros((4, 6), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="one device"):
        snr.matmul_int8(a, sa, w.to("meta"), sw)
    with pytest.raises(ValueError, match="CUDA tensors"):
        snr.matmul_int8(a, sa, w, sw)
