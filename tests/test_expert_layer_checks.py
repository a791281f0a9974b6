"""Refusals of the calls around the experts (FP8 boundaries and products, sorting, gathering, combining,
activation), in the C ABI (before any CUDA call) and in the binding: no GPU."""
from __future__ import annotations

import ctypes

import pytest
import torch

import sandwich_norm_residual_gb300 as snr
from sandwich_norm_residual_gb300 import _lib, build

A = 0x7F0000000000  # fake device addresses: never dereferenced
D = 5120
NO_DEVICE = (_lib.BEAM_ERR_CUDA, _lib.BEAM_ERR_DEVICE)
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_boundary_fp8_argument_errors(lib):
    H, X, PW, QW, Q, S, E, W = (A + (i << 32) for i in range(8))

    def dense(T=4, d=D, n=2, eps=1e-6, h=H, x=X, q=Q, s=S, opts=None):
        return lib.beam_boundary_fused_fp8(None, h, x, PW, QW, n, eps, T, d, q, s, opts)

    def moe(T=4, d=D, h=H, e=E, w=W, rs=1.0, q=Q, s=S, opts=None):
        return lib.beam_moe_combine_boundary_fp8(None, h, e, w, rs, PW, QW, 2, 1e-6, T, d, q, s, opts)

    for call in (dense, moe):
        assert call(d=12) == _lib.BEAM_ERR_SHAPE
        assert call(T=-1) == _lib.BEAM_ERR_SHAPE
        assert call(T=0, h=None, q=None, s=None) == _lib.BEAM_OK
        assert call(h=None) == _lib.BEAM_ERR_NULL
        assert call(q=None) == _lib.BEAM_ERR_NULL
        assert call(s=None) == _lib.BEAM_ERR_NULL
        assert call(q=Q + 8) == _lib.BEAM_ERR_ALIGN
        assert call(s=S + 4) == _lib.BEAM_ERR_ALIGN
        assert call(s=Q + 4 * D - 16) == _lib.BEAM_ERR_ALIAS           # scales over the codes
        assert call(s=H - 4 * 4 * (D // 128) + 16) == _lib.BEAM_ERR_ALIAS  # the last row's scales in h
        assert call(q=H + 64) == _lib.BEAM_ERR_ALIAS
        ring = _lib.LaunchOpts(stages=2)
        assert call(opts=ctypes.byref(ring)) == _lib.BEAM_ERR_ARG
        assert call() in NO_DEVICE
    assert dense(n=0) == _lib.BEAM_ERR_ARG
    assert dense(x=H + 2 * D) == _lib.BEAM_ERR_ALIAS
    assert moe(rs=float("nan")) == _lib.BEAM_ERR_ARG
    assert moe(q=W) == _lib.BEAM_ERR_ALIAS


def test_product_argument_errors(lib):
    AA, AS, W, WS, O, F = (A + (i << 40) for i in range(6))

    def mm(M=4, N=40, K=64, a=AA, sa=AS, w=W, sw=WS, ty=0, o=O, flags=0):
        return lib.beam_matmul_fp8(None, a, sa, w, sw, M, N, K, ty, o, flags)

    def ex(R=4, E=3, N=40, K=64, a=AA, sa=AS, off=F, w=W, sw=WS, ty=0, o=O, flags=0):
        return lib.beam_matmul_fp8_experts(None, a, sa, off, w, sw, R, E, N, K, ty, o, flags)

    for call, rows in ((mm, "M"), (ex, "R")):
        for bad in (-1, _lib.BEAM_MATMUL_FP8_MAX_ROWS + 1):
            assert call(**{rows: bad}) == _lib.BEAM_ERR_SHAPE
        assert call(N=-1) == _lib.BEAM_ERR_SHAPE
        for K in (0, 8, 24, -16, _lib.BEAM_MATMUL_MAX_K + 16):
            assert call(K=K) == _lib.BEAM_ERR_SHAPE
        # more tiles than 31 bits count
        assert call(**{rows: _lib.BEAM_MATMUL_FP8_MAX_ROWS}, N=1 << 14, K=16) == _lib.BEAM_ERR_SHAPE
        assert call(ty=2) == _lib.BEAM_ERR_ARG
        assert call(flags=_lib.BEAM_OPT_PDL) == _lib.BEAM_ERR_ARG
        assert call(flags=_lib.BEAM_OPT_TEST_WAIT_TIMEOUT) == _lib.BEAM_ERR_ARG  # K = 64: no second 128
        assert call(**{rows: 0}, a=None) == _lib.BEAM_OK
        assert call(N=0, w=None) == _lib.BEAM_OK
        for name in ("a", "sa", "w", "sw", "o"):
            assert call(**{name: None}) == _lib.BEAM_ERR_NULL
        assert call(a=AA + 8) == _lib.BEAM_ERR_ALIGN
        assert call(w=W + 4) == _lib.BEAM_ERR_ALIGN
        assert call(sa=AS + 2) == _lib.BEAM_ERR_ALIGN
        assert call(o=O + 1) == _lib.BEAM_ERR_ALIGN
        assert call(o=O + 2, ty=1) == _lib.BEAM_ERR_ALIGN
        assert call(o=AA + 64) == _lib.BEAM_ERR_ALIAS
        assert call(o=W - 2) == _lib.BEAM_ERR_ALIAS
        assert call(o=AS + 4) == _lib.BEAM_ERR_ALIAS
        assert call(o=WS) == _lib.BEAM_ERR_ALIAS
        assert call(o=O + 2) in NO_DEVICE
    assert ex(E=0) == _lib.BEAM_ERR_SHAPE and ex(E=_lib.BEAM_MOE_MAX_EXPERTS + 1) == _lib.BEAM_ERR_SHAPE
    assert ex(off=None) == _lib.BEAM_ERR_NULL
    assert ex(off=F + 2) == _lib.BEAM_ERR_ALIGN
    assert ex(o=F) == _lib.BEAM_ERR_ALIAS
    assert ex(o=W + 3 * 40 * 64 - 2) == _lib.BEAM_ERR_ALIAS  # the last expert's channels


def test_sort_argument_errors(lib):
    I, F, S, P = (A + (i << 40) for i in range(4))
    need = lib.beam_moe_sort_workspace

    def sort(T=4, k=8, E=256, i=I, f=F, s=S, ws=P, nb=1 << 30):
        return lib.beam_moe_sort(None, i, T, k, E, f, s, ws, nb)

    for bad in (dict(T=-1), dict(k=0), dict(k=17), dict(E=0), dict(E=513), dict(T=_lib.BEAM_MOE_MAX_PAIRS // 8 + 1)):
        assert sort(**bad) == _lib.BEAM_ERR_SHAPE
        assert need(bad.get("T", 4), bad.get("k", 8), bad.get("E", 256)) == -1
    assert need(4, 8, 256) == 0 and need(16384, 8, 256) > 0
    big = dict(T=16384)
    assert sort(nb=need(16384, 8, 256) - 1, **big) == _lib.BEAM_ERR_ARG
    assert sort(ws=None, **big) == _lib.BEAM_ERR_NULL
    assert sort(ws=P + 4, **big) == _lib.BEAM_ERR_ALIGN
    assert sort(ws=S + 16, **big) == _lib.BEAM_ERR_ALIAS
    for name in ("i", "f", "s"):
        assert sort(**{name: None}) == _lib.BEAM_ERR_NULL
        assert sort(**{name: A + (7 << 40) + 2}) == _lib.BEAM_ERR_ALIGN
    assert sort(T=0, i=None, s=None, f=None) == _lib.BEAM_ERR_NULL  # offsets are written for no tokens too
    assert sort(s=I + 4) == _lib.BEAM_ERR_ALIAS
    assert sort(f=S + 8) == _lib.BEAM_ERR_ALIAS
    assert sort(ws=None, nb=0) in NO_DEVICE


def test_gather_argument_errors(lib):
    X, C, S, O, P = (A + (i << 40) for i in range(5))

    def gather(x=X, rb=D, c=C, cb=160, s=S, T=4, k=8, R=32, o=O, p=P):
        return lib.beam_moe_gather(None, x, rb, c, cb, s, T, k, R, o, p)

    for bad in (dict(rb=0), dict(rb=6), dict(rb=4 * _lib.BEAM_MAX_D + 4), dict(cb=-4), dict(cb=2), dict(k=0), dict(k=17),
                dict(T=-1), dict(R=-1), dict(R=_lib.BEAM_MOE_MAX_PAIRS + 1)):
        assert gather(**bad) == _lib.BEAM_ERR_SHAPE
    assert gather(T=0, x=None, o=None) == _lib.BEAM_OK
    for name in ("x", "c", "s", "o", "p"):
        assert gather(**{name: None}) == _lib.BEAM_ERR_NULL
        assert gather(**{name: A + (7 << 40) + 2}) == _lib.BEAM_ERR_ALIGN
    assert gather(c=None, p=None, cb=0) in NO_DEVICE
    assert gather(o=X + 16) == _lib.BEAM_ERR_ALIAS
    assert gather(p=O + 32 * D - 4) == _lib.BEAM_ERR_ALIAS
    assert gather(o=S) == _lib.BEAM_ERR_ALIAS
    assert gather(x=X + 4, o=O + 4) in NO_DEVICE


def test_combine_argument_errors(lib):
    X, R_, S, W, O, DW = (A + (i << 40) for i in range(6))

    def back(d=R_, s=S, T=4, k=8, R=32, dim=D, ty=0, o=O):
        return lib.beam_moe_gather_backward(None, d, s, T, k, R, dim, ty, o)

    def combine(d=R_, s=S, w=W, T=4, k=8, R=32, dim=D, ty=0, o=O):
        return lib.beam_moe_combine(None, d, s, w, T, k, R, dim, ty, o)

    def grad(x=X, d=R_, s=S, w=W, T=4, k=8, R=32, dim=D, ty=0, o=O, dw=DW):
        return lib.beam_moe_combine_backward(None, x, d, s, w, T, k, R, dim, ty, o, dw)

    for call in (back, combine, grad):
        for bad in (dict(T=-1), dict(k=0), dict(k=17), dict(R=-1), dict(dim=0), dict(dim=12),
                    dict(dim=_lib.BEAM_MAX_D + 8)):
            assert call(**bad) == _lib.BEAM_ERR_SHAPE
        assert call(ty=2) == _lib.BEAM_ERR_ARG
        assert call(T=0, d=None, s=None, o=None) == _lib.BEAM_OK
        for name in ("d", "s", "o"):
            assert call(**{name: None}) == _lib.BEAM_ERR_NULL
        assert call(d=R_ + 8) == _lib.BEAM_ERR_ALIGN and call(o=O + 4) == _lib.BEAM_ERR_ALIGN
        assert call(s=S + 2) == _lib.BEAM_ERR_ALIGN
        assert call(o=R_ + 16) == _lib.BEAM_ERR_ALIAS and call(o=S) == _lib.BEAM_ERR_ALIAS
        assert call() in NO_DEVICE and call(ty=1) in NO_DEVICE
    assert combine(w=None) == _lib.BEAM_ERR_NULL and combine(w=W + 2) == _lib.BEAM_ERR_ALIGN
    assert combine(o=W) == _lib.BEAM_ERR_ALIAS
    for name in ("x", "w", "dw"):
        assert grad(**{name: None}) == _lib.BEAM_ERR_NULL
    assert grad(x=X + 8) == _lib.BEAM_ERR_ALIGN and grad(dw=DW + 2) == _lib.BEAM_ERR_ALIGN
    assert grad(o=X) == _lib.BEAM_ERR_ALIAS and grad(dw=O + 64) == _lib.BEAM_ERR_ALIAS and grad(dw=W) == _lib.BEAM_ERR_ALIAS


def test_swiglu_argument_errors(lib):
    X, L, Q, S = (A + (i << 40) for i in range(4))

    def act(x=X, live=L, R=8, F=2560, q=Q, s=S):
        return lib.beam_swiglu_fp8(None, x, live, R, F, q, s)

    for bad in (dict(R=-1), dict(R=_lib.BEAM_MOE_MAX_PAIRS + 1), dict(F=0), dict(F=24), dict(F=_lib.BEAM_MATMUL_MAX_K + 16)):
        assert act(**bad) == _lib.BEAM_ERR_SHAPE
    assert act(R=0, x=None) == _lib.BEAM_OK
    for name in ("x", "q", "s"):
        assert act(**{name: None}) == _lib.BEAM_ERR_NULL
    assert act(x=X + 8) == _lib.BEAM_ERR_ALIGN and act(q=Q + 4) == _lib.BEAM_ERR_ALIGN
    assert act(s=S + 2) == _lib.BEAM_ERR_ALIGN and act(live=L + 2) == _lib.BEAM_ERR_ALIGN
    assert act(q=X + 64) == _lib.BEAM_ERR_ALIAS and act(s=Q) == _lib.BEAM_ERR_ALIAS and act(s=L) == _lib.BEAM_ERR_ALIAS
    assert act(live=None) in NO_DEVICE


# ---------------------------------------------------------------- the binding

def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def f8(*shape):
    return torch.zeros(shape, dtype=torch.uint8).view(FP8)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_binding_checks_the_fp8_boundaries():
    T, d = 4, 264
    h, x, w = bf(T, d), bf(T, d), bf(d)
    with pytest.raises(ValueError, match="y_fp8 must have shape"):
        snr.boundary_fused_fp8(h, x, w, w, 2, y_fp8=f8(T, d - 8))
    with pytest.raises(ValueError, match="y_scale must have shape"):
        snr.boundary_fused_fp8(h, x, w, w, 2, y_scale=torch.zeros(T, 2))
    with pytest.raises(TypeError, match="y_fp8 must be"):
        snr.boundary_fused_fp8(h, x, w, w, 2, y_fp8=torch.zeros((T, d), dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA tensors"):
        snr.boundary_fused_fp8(h, x, w, w, 2)
    e, tw = bf(T, 8, d), torch.zeros((T, 8))
    with pytest.raises(ValueError, match="shape mismatch"):
        snr.moe_combine_boundary_fp8(h, e[:3].contiguous(), tw, w, w, 2)
    with pytest.raises(ValueError, match="one device"):
        snr.moe_combine_boundary_fp8(h, e, tw.to("meta"), w, w, 2)


def test_binding_checks_the_products():
    a, sa, w, sw = f8(4, 272), torch.zeros(4, 3), f8(130, 272), torch.zeros(2, 3)
    with pytest.raises(ValueError, match="rows of"):
        snr.matmul_fp8(a, sa, f8(130, 256), sw)
    with pytest.raises(ValueError, match="a_scale must have shape"):
        snr.matmul_fp8(a, torch.zeros(4, 2), w, sw)
    with pytest.raises(ValueError, match="w_scale must have shape"):
        snr.matmul_fp8(a, sa, w, torch.zeros(130, 3))
    with pytest.raises(TypeError, match="a must be"):
        snr.matmul_fp8(a.view(torch.uint8), sa, w, sw)
    with pytest.raises(TypeError, match="w must be"):
        snr.matmul_fp8(a, sa, w.view(torch.uint8).view(torch.float8_e5m2), sw)
    with pytest.raises(ValueError, match="contiguous"):
        snr.matmul_fp8(a, sa, f8(272, 130).t(), sw)
    with pytest.raises(TypeError, match="out_dtype"):
        snr.matmul_fp8(a, sa, w, sw, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="out must have shape"):
        snr.matmul_fp8(a, sa, w, sw, out=bf(4, 131))
    with pytest.raises(ValueError, match="one device"):
        snr.matmul_fp8(a, sa, w.to("meta"), sw)
    with pytest.raises(ValueError, match="CUDA tensors"):
        snr.matmul_fp8(a, sa, w, sw)
    we, swe, off = f8(3, 130, 272), torch.zeros(3, 2, 3), i32(4)
    with pytest.raises(ValueError, match="offsets must have shape"):
        snr.matmul_fp8_experts(a, sa, i32(3), we, swe)
    with pytest.raises(TypeError, match="offsets must be"):
        snr.matmul_fp8_experts(a, sa, None, we, swe)
    with pytest.raises(TypeError, match="offsets must be"):
        snr.matmul_fp8_experts(a, sa, off.long(), we, swe)
    with pytest.raises(ValueError, match="w_scale must have shape"):
        snr.matmul_fp8_experts(a, sa, off, we, swe[:2].contiguous())
    with pytest.raises(ValueError, match="3-d"):
        snr.matmul_fp8_experts(a, sa, off, w, swe)
    with pytest.raises(ValueError, match="CUDA tensors"):
        snr.matmul_fp8_experts(a, sa, off, we, swe)


def test_binding_checks_sorting_and_gathering():
    idx = i32(6, 4)
    with pytest.raises(TypeError, match="topk_idx must be"):
        snr.moe_sort(idx.long(), 8)
    with pytest.raises(ValueError, match="at least 1"):
        snr.moe_sort(idx, 0)
    with pytest.raises(ValueError, match="offsets must have shape"):
        snr.moe_sort(idx, 8, offsets=i32(8))
    with pytest.raises(ValueError, match="slots must have shape"):
        snr.moe_sort(idx, 8, slots=i32(6, 3))
    with pytest.raises(ValueError, match="CUDA tensors"):
        snr.moe_sort(idx, 8)
    x, slots, sc = bf(6, 16), i32(6, 4), torch.zeros(6, 2)
    with pytest.raises(ValueError, match="shape mismatch"):
        snr.moe_gather(x, i32(5, 4))
    with pytest.raises(ValueError, match="scale must have shape"):
        snr.moe_gather(x, slots, scale=sc[:5].contiguous())
    with pytest.raises(TypeError, match="scale must be"):
        snr.moe_gather(x, slots, scale=sc.double())
    with pytest.raises(ValueError, match="1-d or 2-d"):
        snr.moe_gather(x, slots, scale=torch.zeros(6, 2, 2))
    with pytest.raises(ValueError, match="out_scale without scale"):
        snr.moe_gather(x, slots, out_scale=torch.zeros(24, 2))
    with pytest.raises(ValueError, match="out_scale must have shape"):
        snr.moe_gather(x, slots, scale=sc, out_scale=torch.zeros(24, 3))
    with pytest.raises(ValueError, match="out must have shape"):
        snr.moe_gather(x, slots, out=bf(24, 8))
    with pytest.raises(TypeError, match="out must be"):
        snr.moe_gather(x, slots, out=torch.zeros(24, 16))
    with pytest.raises(ValueError, match="contiguous"):
        snr.moe_gather(bf(16, 6).t(), slots)
    with pytest.raises(ValueError, match="CUDA tensors"):
        snr.moe_gather(x, slots, scale=sc)


def test_binding_checks_combining():
    rows, slots, w = bf(24, 16), i32(6, 4), torch.zeros(6, 4)
    with pytest.raises(TypeError, match="rows must be"):
        snr.moe_combine(rows.half(), slots, w)
    with pytest.raises(TypeError, match="topk_w must be"):
        snr.moe_combine(rows, slots, None)
    with pytest.raises(ValueError, match="topk_w must have shape"):
        snr.moe_combine(rows, slots, w[:, :3].contiguous())
    with pytest.raises(TypeError, match="slots must be"):
        snr.moe_combine(rows, slots.long(), w)
    with pytest.raises(ValueError, match="out must have shape"):
        snr.moe_combine(rows, slots, w, out=bf(5, 16))
    with pytest.raises(TypeError, match="dx must be"):
        snr.moe_gather_backward(rows, slots, dx=torch.zeros(6, 16))
    with pytest.raises(ValueError, match="CUDA tensors"):
        snr.moe_combine(rows, slots, w)
    dx = bf(6, 16)
    with pytest.raises(ValueError, match="dx must have shape"):
        snr.moe_combine_backward(bf(6, 8), rows, slots, w)
    with pytest.raises(TypeError, match="dx must be"):
        snr.moe_combine_backward(dx.float(), rows, slots, w)
    with pytest.raises(ValueError, match="drows must have shape"):
        snr.moe_combine_backward(dx, rows, slots, w, drows=bf(23, 16))
    with pytest.raises(ValueError, match="dw must have shape"):
        snr.moe_combine_backward(dx, rows, slots, w, dw=torch.zeros(6, 3))
    with pytest.raises(ValueError, match="one device"):
        snr.moe_combine_backward(dx, rows, slots.to("meta"), w)


def test_binding_checks_the_activation():
    with pytest.raises(TypeError, match="gate_up must be"):
        snr.swiglu_fp8(torch.zeros(4, 64))
    with pytest.raises(ValueError, match="even number"):
        snr.swiglu_fp8(bf(4, 33))
    with pytest.raises(ValueError, match="at least one"):
        snr.swiglu_fp8(bf(4, 64), offsets=i32(0))
    with pytest.raises(TypeError, match="offsets must be"):
        snr.swiglu_fp8(bf(4, 64), offsets=torch.zeros(3))
    with pytest.raises(ValueError, match="y_fp8 must have shape"):
        snr.swiglu_fp8(bf(4, 64), y_fp8=f8(4, 64))
    with pytest.raises(ValueError, match="y_scale must have shape"):
        snr.swiglu_fp8(bf(4, 64), y_scale=torch.zeros(4, 2))
    with pytest.raises(ValueError, match="CUDA tensors"):
        snr.swiglu_fp8(bf(4, 64), offsets=i32(3))


def test_none_where_a_tensor_belongs_is_refused():
    for call in (lambda: snr.matmul_fp8(None, None, None, None), lambda: snr.moe_sort(None, 4),
                 lambda: snr.moe_gather(None, None), lambda: snr.moe_combine(None, None, torch.zeros(1, 1)),
                 lambda: snr.swiglu_fp8(None), lambda: snr.boundary_fused_fp8(None, None, None, None, 1)):
        with pytest.raises((TypeError, ValueError)):
            call()
