"""Fused sublayer boundary of the Beam decoder on GB300 (sm_103a).

Python binding of ``libbeamboundary`` (C ABI: ``include/beam_boundary.h``).
This module only marshals torch CUDA tensors into the C calls; every step of
the boundary runs in the library's CUDA kernels. There is no CPU or PyTorch
fallback: without the built library, calls raise ``ImportError``.

    y = boundary_fused(h, x, post_w, pre_w, n, eps)          # h updated in place
    y = moe_combine_boundary(h, expert_out, topk_w, post_w, pre_w, n, eps)

Every call takes ``stream`` (default: the current stream). Operands that other streams write
must be ready on it, and are kept (or recorded on it) until it is done with them. Outputs that
the caller does not give come from the memory pool of that stream, as any tensor made under
``torch.cuda.stream(stream)``: before another stream reads one, make it wait for ``stream``, and
let it ``record_stream`` what is freed before it is done.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

from . import _lib
from ._lib import LaunchOpts  # noqa: F401

__all__ = ["boundary_fused", "moe_combine_boundary", "boundary_fused_host",
           "moe_combine_boundary_host", "boundary_fused_nvfp4",
           "moe_combine_boundary_nvfp4", "boundary_fused_int8", "moe_combine_boundary_int8",
           "boundary_fused_fp8", "moe_combine_boundary_fp8",
           "matmul_int8", "matmul_fp8", "matmul_fp8_experts", "swiglu_fp8",
           "moe_sort", "moe_gather", "moe_gather_backward", "moe_combine", "moe_combine_backward",
           "moe_route", "moe_balance_loss", "moe_balance_loss_backward",
           "router_sigmoid", "qk_norm", "sync_status",
           "exact_sum_count",
           "version", "BeamError", "LaunchOpts", "library"]


class BeamError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.load().beam_status_string(status).decode()
        super().__init__(f"{where}: status {status} ({msg})")


def library() -> ctypes.CDLL:
    """The loaded ``libbeamboundary.so`` (raises ImportError when it is not built)."""
    return _lib.load()


def _stream_ptr(stream) -> int | None:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream or None


def _check(t, name: str, dtype, ndim: int):
    """Type, dtype, rank and layout of one operand (devices: ``_on_current_device``)."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.dim() != ndim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-d tensor")


def _shape(t, name: str, shape: tuple):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")


def _on_current_device(**tensors):
    """Every operand on one CUDA device, the current one: the library launches on the
    current device and takes the pointers as they are, so a tensor elsewhere would
    reach the kernel as a foreign address. Checked after the shapes, before any launch."""
    import torch
    devs = {name: t.device for name, t in tensors.items()}
    if len(set(devs.values())) != 1:
        raise ValueError("operands must all be on one device: "
                         + ", ".join(f"{n} on {d}" for n, d in devs.items()))
    dev = next(iter(devs.values()))
    if dev.type != "cuda":
        raise ValueError(f"operands must be CUDA tensors (got {dev})")
    cur = torch.cuda.current_device()
    if dev.index != cur:
        raise ValueError(f"operands are on {dev} but the current device is cuda:{cur}: "
                         f"call under `with torch.cuda.device({dev.index}):`")


_torch = None


def _dims(t, n: int):
    """The shape of an n-d tensor, or n times -1 (which no operand has) for anything else."""
    shape = getattr(t, "shape", ())
    return shape if len(shape) == n else (-1,) * n


def _ready(*operands) -> bool:
    """Whether every (tensor, dtype, shape) is as said, contiguous and on the current CUDA
    device. The calls whose kernels take microseconds ask this first, in one cheap pass, and
    look for what is wrong only when it says no."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    Tensor, dev = _torch.Tensor, None
    for t, dtype, shape in operands:
        if not (isinstance(t, Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous()):
            return False
        d = t.get_device()
        if dev is None:
            dev = d
        if d != dev or d < 0:
            return False
    return dev == _torch._C._cuda_getDevice()  # initialised: the operands are CUDA tensors


def _raw_stream(stream, t) -> int | None:
    """The stream's handle, without a stream object for the current one."""
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(t.get_device()) or None
    return stream.cuda_stream or None


_HERE = contextlib.nullcontext()


def _pool(stream):
    """A context in which tensors come from the memory pool of the stream that the call runs on.
    Another stream's pool may hand out memory that work queued there still reads or writes, and
    takes it back for such work when it is freed. Entering a stream takes 10 us, so only where
    it is not the current one."""
    import torch
    if stream is None:
        return _HERE
    if not hasattr(stream, "device_index"):  # anything that carries a handle is a stream here
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    if stream.cuda_stream == torch._C._cuda_getCurrentRawStream(stream.device_index):
        return _HERE
    return torch.cuda.stream(stream)


def _workspace(nbytes: int, device):
    """Device memory for one call (within ``_pool``): freed at the call's end, it goes to later
    work of the call's stream alone. None for no bytes."""
    import torch
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _c_int(v) -> int:
    """A number that the C ABI takes as int (ctypes would cut it to its low 32 bits)."""
    v = int(v)
    if not -0x80000000 <= v <= 0x7FFFFFFF:
        raise ValueError(f"{v} is more than a 32-bit argument holds")
    return v


def _opts(opts):
    if opts is None:
        return None
    if isinstance(opts, dict):
        opts = LaunchOpts(**opts)
    return ctypes.byref(opts)


def boundary_fused(h, x, post_w, pre_w, n: int, eps: float = 1e-6, y=None, stream=None, opts=None):
    """Dense boundary on torch CUDA tensors; updates ``h`` in place and returns ``y``.

    h, x: [T, D] bfloat16; post_w, pre_w: [D] bfloat16; n >= 1 (index of the residual add).
    """
    import torch
    _check(h, "h", torch.bfloat16, 2)
    _check(x, "x", torch.bfloat16, 2)
    _check(post_w, "post_w", torch.bfloat16, 1)
    _check(pre_w, "pre_w", torch.bfloat16, 1)
    T, D = h.shape
    if x.shape != h.shape or post_w.shape[0] != D or pre_w.shape[0] != D:
        raise ValueError("shape mismatch: h, x [T, D]; post_w, pre_w [D]")
    if y is None:
        with _pool(stream):
            y = torch.empty_like(h)
    _check(y, "y", torch.bfloat16, 2)
    _shape(y, "y", (T, D))
    _on_current_device(h=h, x=x, post_w=post_w, pre_w=pre_w, y=y)
    lib = _lib.load()
    args = (_stream_ptr(stream), h.data_ptr(), x.data_ptr(), post_w.data_ptr(), pre_w.data_ptr(),
            _c_int(n), float(eps), T, _c_int(D), y.data_ptr())
    st = lib.beam_boundary_fused(*args) if opts is None else lib.beam_boundary_fused_ex(
        *args, _opts(opts))
    if st != 0:
        raise BeamError(st, "beam_boundary_fused")
    return y


def moe_combine_boundary(h, expert_out, topk_w, post_w, pre_w, n: int, eps: float = 1e-6, y=None,
                         stream=None, opts=None, route_scale: float | None = None):
    """MoE boundary: combine the top-8 expert outputs with FP32 weights, then the dense boundary.

    h: [T, D] bf16; expert_out: [T, 8, D] bf16; topk_w: [T, 8] float32 with the routing
    scale included, or, when ``route_scale`` is given, without it (the kernel then applies
    it to the combined sum).
    """
    import torch
    _check(h, "h", torch.bfloat16, 2)
    _check(expert_out, "expert_out", torch.bfloat16, 3)
    _check(topk_w, "topk_w", torch.float32, 2)
    _check(post_w, "post_w", torch.bfloat16, 1)
    _check(pre_w, "pre_w", torch.bfloat16, 1)
    T, D = h.shape
    K = _lib.BEAM_MOE_TOPK
    if expert_out.shape != (T, K, D) or topk_w.shape != (T, K):
        raise ValueError(f"shape mismatch: expert_out [T, {K}, D], topk_w [T, {K}]")
    if post_w.shape[0] != D or pre_w.shape[0] != D:
        raise ValueError("shape mismatch: post_w, pre_w [D]")
    if y is None:
        with _pool(stream):
            y = torch.empty_like(h)
    _check(y, "y", torch.bfloat16, 2)
    _shape(y, "y", (T, D))
    _on_current_device(h=h, expert_out=expert_out, topk_w=topk_w, post_w=post_w, pre_w=pre_w, y=y)
    lib = _lib.load()
    if route_scale is not None:
        if opts is not None:
            raise ValueError("route_scale and opts cannot be combined")
        st = lib.beam_moe_combine_boundary_scaled(
            _stream_ptr(stream), h.data_ptr(), expert_out.data_ptr(), topk_w.data_ptr(),
            float(route_scale), post_w.data_ptr(), pre_w.data_ptr(), _c_int(n), float(eps), T, _c_int(D),
            y.data_ptr())
        if st != 0:
            raise BeamError(st, "beam_moe_combine_boundary_scaled")
        return y
    args = (_stream_ptr(stream), h.data_ptr(), expert_out.data_ptr(), topk_w.data_ptr(),
            post_w.data_ptr(), pre_w.data_ptr(), _c_int(n), float(eps), T, _c_int(D), y.data_ptr())
    st = lib.beam_moe_combine_boundary(*args) if opts is None else \
        lib.beam_moe_combine_boundary_ex(*args, _opts(opts))
    if st != 0:
        raise BeamError(st, "beam_moe_combine_boundary")
    return y


def _check_any(t, name: str, dtype, ndim: int):
    """A CUDA tensor or a CPU tensor (page-locked, or pageable where the device
    reads pageable memory: the library decides)."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type not in ("cuda", "cpu"):
        raise ValueError(f"{name} must be a CUDA or CPU tensor (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.dim() != ndim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-d tensor")


def _like_host(h, stream):
    import torch
    if h.device.type == "cuda":
        with _pool(stream):
            return torch.empty_like(h)
    return torch.empty(h.shape, dtype=h.dtype, pin_memory=True)


def boundary_fused_host(h, x, post_w, pre_w, n: int, eps: float = 1e-6, y=None, stream=None):
    """Dense boundary on a batch in host memory: h, x, y (and the weights) may be
    page-locked CPU tensors (``tensor.pin_memory()``), read and written by the kernels
    over the CPU-GPU link. Asynchronous on ``stream`` (default: the current CUDA
    stream): synchronise before touching the host tensors. Returns y (page-locked
    CPU when h is on the CPU)."""
    import torch
    _check_any(h, "h", torch.bfloat16, 2)
    _check_any(x, "x", torch.bfloat16, 2)
    _check_any(post_w, "post_w", torch.bfloat16, 1)
    _check_any(pre_w, "pre_w", torch.bfloat16, 1)
    T, D = h.shape
    if x.shape != h.shape or post_w.shape[0] != D or pre_w.shape[0] != D:
        raise ValueError("shape mismatch: h, x [T, D]; post_w, pre_w [D]")
    if y is None:
        y = _like_host(h, stream)
    _check_any(y, "y", torch.bfloat16, 2)
    _shape(y, "y", (T, D))
    st = _lib.load().beam_boundary_fused_host(_stream_ptr(stream), h.data_ptr(), x.data_ptr(),
                                              post_w.data_ptr(), pre_w.data_ptr(), _c_int(n),
                                              float(eps), T, _c_int(D), y.data_ptr())
    if st != 0:
        raise BeamError(st, "beam_boundary_fused_host")
    return y


def moe_combine_boundary_host(h, expert_out, topk_w, post_w, pre_w, n: int, eps: float = 1e-6,
                              y=None, stream=None):
    """MoE boundary on a batch in host memory (see ``boundary_fused_host``)."""
    import torch
    _check_any(h, "h", torch.bfloat16, 2)
    _check_any(expert_out, "expert_out", torch.bfloat16, 3)
    _check_any(topk_w, "topk_w", torch.float32, 2)
    _check_any(post_w, "post_w", torch.bfloat16, 1)
    _check_any(pre_w, "pre_w", torch.bfloat16, 1)
    T, D = h.shape
    K = _lib.BEAM_MOE_TOPK
    if (expert_out.shape != (T, K, D) or topk_w.shape != (T, K) or post_w.shape[0] != D
            or pre_w.shape[0] != D):
        raise ValueError(f"shape mismatch: h [T, D]; expert_out [T, {K}, D]; topk_w [T, {K}]")
    if y is None:
        y = _like_host(h, stream)
    _check_any(y, "y", torch.bfloat16, 2)
    _shape(y, "y", (T, D))
    st = _lib.load().beam_moe_combine_boundary_host(
        _stream_ptr(stream), h.data_ptr(), expert_out.data_ptr(), topk_w.data_ptr(),
        post_w.data_ptr(), pre_w.data_ptr(), _c_int(n), float(eps), T, _c_int(D), y.data_ptr())
    if st != 0:
        raise BeamError(st, "beam_moe_combine_boundary_host")
    return y


def _nvfp4_out(h, q, sf, stream):
    import torch
    T, D = h.shape
    if D % 16:
        raise ValueError("NVFP4 output needs D to be a multiple of 16")
    with _pool(stream):
        if q is None:
            q = torch.empty((T, D // 2), dtype=torch.uint8, device=h.device)
        if sf is None:
            sf = torch.empty((T, D // 16), dtype=torch.uint8, device=h.device)
    _check(q, "y_fp4", torch.uint8, 2)
    _check(sf, "y_scale", torch.uint8, 2)
    if tuple(q.shape) != (T, D // 2) or tuple(sf.shape) != (T, D // 16):
        raise ValueError("shape mismatch: y_fp4 [T, D/2]; y_scale [T, D/16]")
    return q, sf


def boundary_fused_nvfp4(h, x, post_w, pre_w, n: int, eps: float, y_global_scale: float,
                         y_fp4=None, y_scale=None, stream=None, opts=None):
    """Dense boundary with y as NVFP4; updates h in place, returns (y_fp4 [T, D/2] uint8,
    y_scale [T, D/16] uint8)."""
    import torch
    for t, name in ((h, "h"), (x, "x")):
        _check(t, name, torch.bfloat16, 2)
    _check(post_w, "post_w", torch.bfloat16, 1)
    _check(pre_w, "pre_w", torch.bfloat16, 1)
    T, D = h.shape
    if x.shape != h.shape or post_w.shape[0] != D or pre_w.shape[0] != D:
        raise ValueError("shape mismatch: h, x [T, D]; post_w, pre_w [D]")
    q, sf = _nvfp4_out(h, y_fp4, y_scale, stream)
    _on_current_device(h=h, x=x, post_w=post_w, pre_w=pre_w, y_fp4=q, y_scale=sf)
    st = _lib.load().beam_boundary_fused_nvfp4(_stream_ptr(stream), h.data_ptr(), x.data_ptr(),
                                               post_w.data_ptr(), pre_w.data_ptr(), _c_int(n),
                                               float(eps), T, _c_int(D), float(y_global_scale),
                                               q.data_ptr(), sf.data_ptr(), _opts(opts))
    if st != 0:
        raise BeamError(st, "beam_boundary_fused_nvfp4")
    return q, sf


def moe_combine_boundary_nvfp4(h, expert_out, topk_w, post_w, pre_w, n: int, eps: float,
                               y_global_scale: float, y_fp4=None, y_scale=None, stream=None,
                               opts=None):
    """MoE boundary with y as NVFP4; updates h in place, returns (y_fp4, y_scale)."""
    import torch
    _check(h, "h", torch.bfloat16, 2)
    _check(expert_out, "expert_out", torch.bfloat16, 3)
    _check(topk_w, "topk_w", torch.float32, 2)
    _check(post_w, "post_w", torch.bfloat16, 1)
    _check(pre_w, "pre_w", torch.bfloat16, 1)
    T, D = h.shape
    if (expert_out.shape != (T, _lib.BEAM_MOE_TOPK, D) or topk_w.shape != (T, _lib.BEAM_MOE_TOPK)
            or post_w.shape[0] != D or pre_w.shape[0] != D):
        raise ValueError("shape mismatch: h [T, D]; expert_out [T, 8, D]; topk_w [T, 8]")
    q, sf = _nvfp4_out(h, y_fp4, y_scale, stream)
    _on_current_device(h=h, expert_out=expert_out, topk_w=topk_w, post_w=post_w, pre_w=pre_w,
                       y_fp4=q, y_scale=sf)
    st = _lib.load().beam_moe_combine_boundary_nvfp4(
        _stream_ptr(stream), h.data_ptr(), expert_out.data_ptr(), topk_w.data_ptr(),
        post_w.data_ptr(), pre_w.data_ptr(), _c_int(n), float(eps), T, _c_int(D), float(y_global_scale),
        q.data_ptr(), sf.data_ptr(), _opts(opts))
    if st != 0:
        raise BeamError(st, "beam_moe_combine_boundary_nvfp4")
    return q, sf


def _int8_given(q, scale, rows) -> tuple:
    """The caller's outputs, as operands of ``_ready``."""
    if q is None and scale is None:
        return ()
    import torch
    return ((() if q is None else ((q, torch.int8, rows),))
            + (() if scale is None else ((scale, torch.float32, rows[:1]),)))


def _int8_out(h, q, scale, stream, checked: bool):
    import torch
    new_q, new_scale = q is None, scale is None
    with _pool(stream):
        if new_q:
            q = torch.empty(h.shape, dtype=torch.int8, device=h.device)
        if new_scale:
            scale = torch.empty(h.shape[0], dtype=torch.float32, device=h.device)
    if not new_q and not checked:
        _check(q, "y_int8", torch.int8, 2)
        _shape(q, "y_int8", h.shape)
    if not new_scale and not checked:
        _check(scale, "y_scale", torch.float32, 1)
        _shape(scale, "y_scale", h.shape[:1])
    return q, scale


def boundary_fused_int8(h, x, post_w, pre_w, n: int, eps: float = 1e-6, y_int8=None, y_scale=None,
                        stream=None, opts=None):
    """Dense boundary with y as int8 and one FP32 scale per token; updates h in place,
    returns (y_int8 [T, D] int8, y_scale [T] float32), the operands of ``matmul_int8`` (which
    needs D to be a multiple of 16)."""
    import torch
    bf16 = torch.bfloat16
    T, D = rows = _dims(h, 2)
    ready = _ready((h, bf16, rows), (x, bf16, rows), (post_w, bf16, (D,)), (pre_w, bf16, (D,)),
                   *_int8_given(y_int8, y_scale, rows))
    if not ready:
        for t, name in ((h, "h"), (x, "x")):
            _check(t, name, bf16, 2)
        _check(post_w, "post_w", bf16, 1)
        _check(pre_w, "pre_w", bf16, 1)
        if x.shape != h.shape or post_w.shape[0] != D or pre_w.shape[0] != D:
            raise ValueError("shape mismatch: h, x [T, D]; post_w, pre_w [D]")
    q, scale = _int8_out(h, y_int8, y_scale, stream, ready)
    if not ready:
        _on_current_device(h=h, x=x, post_w=post_w, pre_w=pre_w, y_int8=q, y_scale=scale)
    st = _lib.load().beam_boundary_fused_int8(_raw_stream(stream, h), h.data_ptr(), x.data_ptr(),
                                              post_w.data_ptr(), pre_w.data_ptr(), _c_int(n), float(eps), T, _c_int(D),
                                              q.data_ptr(), scale.data_ptr(), _opts(opts))
    if st != 0:
        raise BeamError(st, "beam_boundary_fused_int8")
    return q, scale


def moe_combine_boundary_int8(h, expert_out, topk_w, post_w, pre_w, n: int, eps: float = 1e-6,
                              y_int8=None, y_scale=None, stream=None, opts=None,
                              route_scale: float = 1.0):
    """MoE boundary with y as int8 and one FP32 scale per token; updates h in place, returns
    (y_int8, y_scale). ``route_scale`` multiplies the combined sum (1: topk_w carries it)."""
    import torch
    bf16, K = torch.bfloat16, _lib.BEAM_MOE_TOPK
    T, D = rows = _dims(h, 2)
    ready = _ready((h, bf16, rows), (expert_out, bf16, (T, K, D)), (topk_w, torch.float32, (T, K)),
                   (post_w, bf16, (D,)), (pre_w, bf16, (D,)), *_int8_given(y_int8, y_scale, rows))
    if not ready:
        _check(h, "h", bf16, 2)
        _check(expert_out, "expert_out", bf16, 3)
        _check(topk_w, "topk_w", torch.float32, 2)
        _check(post_w, "post_w", bf16, 1)
        _check(pre_w, "pre_w", bf16, 1)
        if (expert_out.shape != (T, K, D) or topk_w.shape != (T, K) or post_w.shape[0] != D
                or pre_w.shape[0] != D):
            raise ValueError("shape mismatch: h [T, D]; expert_out [T, 8, D]; topk_w [T, 8]")
    q, scale = _int8_out(h, y_int8, y_scale, stream, ready)
    if not ready:
        _on_current_device(h=h, expert_out=expert_out, topk_w=topk_w, post_w=post_w, pre_w=pre_w,
                           y_int8=q, y_scale=scale)
    st = _lib.load().beam_moe_combine_boundary_int8(
        _raw_stream(stream, h), h.data_ptr(), expert_out.data_ptr(), topk_w.data_ptr(),
        float(route_scale), post_w.data_ptr(), pre_w.data_ptr(), _c_int(n), float(eps), T, _c_int(D),
        q.data_ptr(), scale.data_ptr(), _opts(opts))
    if st != 0:
        raise BeamError(st, "beam_moe_combine_boundary_int8")
    return q, scale


def _blocks(n: int) -> int:
    """How many scales n values have."""
    return -(-n // _lib.BEAM_FP8_BLOCK)


def _fp8_given(q, scale, rows) -> tuple:
    """The caller's FP8 outputs, as operands of ``_ready``."""
    if q is None and scale is None:
        return ()
    import torch
    return ((() if q is None else ((q, torch.float8_e4m3fn, rows),))
            + (() if scale is None else ((scale, torch.float32, (rows[0], _blocks(rows[1]))),)))


def _fp8_out(rows, device, q, scale, stream, checked: bool):
    import torch
    new_q, new_scale = q is None, scale is None
    scales = (rows[0], _blocks(rows[1]))
    with _pool(stream):
        if new_q:
            q = torch.empty(rows, dtype=torch.float8_e4m3fn, device=device)
        if new_scale:
            scale = torch.empty(scales, dtype=torch.float32, device=device)
    if not new_q and not checked:
        _check(q, "y_fp8", torch.float8_e4m3fn, 2)
        _shape(q, "y_fp8", rows)
    if not new_scale and not checked:
        _check(scale, "y_scale", torch.float32, 2)
        _shape(scale, "y_scale", scales)
    return q, scale


def boundary_fused_fp8(h, x, post_w, pre_w, n: int, eps: float = 1e-6, y_fp8=None, y_scale=None,
                       stream=None, opts=None):
    """Dense boundary with y as E4M3 and one FP32 scale for each 128 values of a row; updates h in
    place, returns (y_fp8 [T, D] float8_e4m3fn, y_scale [T, ceil(D/128)] float32), the operands of
    ``matmul_fp8`` (which needs D to be a multiple of 16)."""
    import torch
    bf16 = torch.bfloat16
    T, D = rows = _dims(h, 2)
    ready = _ready((h, bf16, rows), (x, bf16, rows), (post_w, bf16, (D,)), (pre_w, bf16, (D,)),
                   *_fp8_given(y_fp8, y_scale, rows))
    if not ready:
        for t, name in ((h, "h"), (x, "x")):
            _check(t, name, bf16, 2)
        _check(post_w, "post_w", bf16, 1)
        _check(pre_w, "pre_w", bf16, 1)
        if x.shape != h.shape or post_w.shape[0] != D or pre_w.shape[0] != D:
            raise ValueError("shape mismatch: h, x [T, D]; post_w, pre_w [D]")
    q, scale = _fp8_out(rows, h.device, y_fp8, y_scale, stream, ready)
    if not ready:
        _on_current_device(h=h, x=x, post_w=post_w, pre_w=pre_w, y_fp8=q, y_scale=scale)
    st = _lib.load().beam_boundary_fused_fp8(_raw_stream(stream, h), h.data_ptr(), x.data_ptr(),
                                             post_w.data_ptr(), pre_w.data_ptr(), _c_int(n), float(eps), T, _c_int(D),
                                             q.data_ptr(), scale.data_ptr(), _opts(opts))
    if st != 0:
        raise BeamError(st, "beam_boundary_fused_fp8")
    return q, scale


def moe_combine_boundary_fp8(h, expert_out, topk_w, post_w, pre_w, n: int, eps: float = 1e-6,
                             y_fp8=None, y_scale=None, stream=None, opts=None,
                             route_scale: float = 1.0):
    """MoE boundary with y as E4M3 and one FP32 scale for each 128 values of a row; updates h in
    place, returns (y_fp8, y_scale). ``route_scale`` multiplies the combined sum (1: topk_w
    carries it)."""
    import torch
    bf16, K = torch.bfloat16, _lib.BEAM_MOE_TOPK
    T, D = rows = _dims(h, 2)
    ready = _ready((h, bf16, rows), (expert_out, bf16, (T, K, D)), (topk_w, torch.float32, (T, K)),
                   (post_w, bf16, (D,)), (pre_w, bf16, (D,)), *_fp8_given(y_fp8, y_scale, rows))
    if not ready:
        _check(h, "h", bf16, 2)
        _check(expert_out, "expert_out", bf16, 3)
        _check(topk_w, "topk_w", torch.float32, 2)
        _check(post_w, "post_w", bf16, 1)
        _check(pre_w, "pre_w", bf16, 1)
        if (expert_out.shape != (T, K, D) or topk_w.shape != (T, K) or post_w.shape[0] != D
                or pre_w.shape[0] != D):
            raise ValueError("shape mismatch: h [T, D]; expert_out [T, 8, D]; topk_w [T, 8]")
    q, scale = _fp8_out(rows, h.device, y_fp8, y_scale, stream, ready)
    if not ready:
        _on_current_device(h=h, expert_out=expert_out, topk_w=topk_w, post_w=post_w, pre_w=pre_w,
                           y_fp8=q, y_scale=scale)
    st = _lib.load().beam_moe_combine_boundary_fp8(
        _raw_stream(stream, h), h.data_ptr(), expert_out.data_ptr(), topk_w.data_ptr(),
        float(route_scale), post_w.data_ptr(), pre_w.data_ptr(), _c_int(n), float(eps), T, _c_int(D),
        q.data_ptr(), scale.data_ptr(), _opts(opts))
    if st != 0:
        raise BeamError(st, "beam_moe_combine_boundary_fp8")
    return q, scale


@functools.lru_cache(maxsize=4096)
def _matmul_workspace(M: int, N: int, K: int) -> int:
    return max(0, _lib.load().beam_matmul_int8_workspace(M, N, K))


def matmul_int8(a, a_scale, w, w_scale, out_dtype=None, out=None, stream=None, pdl: bool = False):
    """Product of int8 tokens and int8 channels, scaled per token and channel.

    a: [M, K] int8 and a_scale: [M] float32, as an int8 boundary writes them; w: [N, K] int8
    and w_scale: [N] float32. K must be a multiple of 16.
    Returns [M, N] in out_dtype: bfloat16 (the default) or float32.
    Integer sums are exact for up to 8 tokens, and for more while no partial sum leaves +-2^24
    (always for K <= 1024); beyond, they carry FP32 roundings and can change with M and N.
    pdl: launch with programmatic dependent launch (BEAM_OPT_PDL), which reads w while kernels
    before it on the stream still run: neither the previous one may write w, nor one in front of
    a chain of calls with pdl (write w; a call with pdl; this call with pdl: w may be read too early).
    """
    import torch
    (M, K), (N, _) = _dims(a, 2), _dims(w, 2)
    if out_dtype is None:
        out_dtype = getattr(out, "dtype", torch.bfloat16)
    ready = _ready((a, torch.int8, (M, K)), (a_scale, torch.float32, (M,)), (w, torch.int8, (N, K)),
                   (w_scale, torch.float32, (N,)), *(() if out is None else ((out, out_dtype, (M, N)),)))
    if not ready:
        _check(a, "a", torch.int8, 2)
        _check(a_scale, "a_scale", torch.float32, 1)
        _check(w, "w", torch.int8, 2)
        _check(w_scale, "w_scale", torch.float32, 1)
        if w.shape[1] != K or a_scale.shape[0] != M or w_scale.shape[0] != N:
            raise ValueError("shape mismatch: a [M, K]; a_scale [M]; w [N, K]; w_scale [N]")
    if out_dtype is not torch.bfloat16 and out_dtype is not torch.float32:
        raise TypeError(f"out_dtype must be bfloat16 or float32 (got {out_dtype})")
    N, K = _c_int(N), _c_int(K)
    ws_bytes = _matmul_workspace(M, N, K)
    with _pool(stream):
        if out is None:
            out = torch.empty((M, N), dtype=out_dtype, device=a.device)
        ws = _workspace(ws_bytes, a.device)
    if not ready:
        _check(out, "out", out_dtype, 2)
        _shape(out, "out", (M, N))
        _on_current_device(a=a, a_scale=a_scale, w=w, w_scale=w_scale, out=out)
    st = _lib.load().beam_matmul_int8(
        _raw_stream(stream, a), a.data_ptr(), a_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(), M, N, K,
        _lib.BEAM_OUT_FP32 if out_dtype is torch.float32 else _lib.BEAM_OUT_BF16, out.data_ptr(),
        ws.data_ptr() if ws_bytes else None, ws_bytes, _lib.BEAM_OPT_PDL if pdl else 0)
    if st != 0:
        raise BeamError(st, "beam_matmul_int8")
    return out


def _fp8_product(a, a_scale, offsets, w, w_scale, out_dtype, out, stream, name: str):
    import torch
    fp8, grouped = torch.float8_e4m3fn, offsets is not None
    M, K = _dims(a, 2)
    E, N = _dims(w, 3)[:2] if grouped else (1, _dims(w, 2)[0])
    experts = (E,) if grouped else ()
    if out_dtype is None:
        out_dtype = getattr(out, "dtype", torch.bfloat16)
    scales = (M, _blocks(K)), (*experts, _blocks(N), _blocks(K))
    ready = _ready((a, fp8, (M, K)), (a_scale, torch.float32, scales[0]), (w, fp8, (*experts, N, K)),
                   (w_scale, torch.float32, scales[1]),
                   *(((offsets, torch.int32, (E + 1,)),) if grouped else ()),
                   *(() if out is None else ((out, out_dtype, (M, N)),)))
    if not ready:
        _check(a, "a", fp8, 2)
        _check(a_scale, "a_scale", torch.float32, 2)
        _check(w, "w", fp8, 3 if grouped else 2)
        _check(w_scale, "w_scale", torch.float32, 3 if grouped else 2)
        if w.shape[-1] != K:
            raise ValueError(f"shape mismatch: a has rows of {K}, w of {w.shape[-1]}")
        _shape(a_scale, "a_scale", scales[0])
        _shape(w_scale, "w_scale", scales[1])
        if grouped:
            _check(offsets, "offsets", torch.int32, 1)
            _shape(offsets, "offsets", (E + 1,))
    if out_dtype is not torch.bfloat16 and out_dtype is not torch.float32:
        raise TypeError(f"out_dtype must be bfloat16 or float32 (got {out_dtype})")
    N, K, E = _c_int(N), _c_int(K), _c_int(E)
    if out is None:
        with _pool(stream):
            out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    if not ready:
        _check(out, "out", out_dtype, 2)
        _shape(out, "out", (M, N))
        _on_current_device(**_given(a=a, a_scale=a_scale, offsets=offsets, w=w, w_scale=w_scale, out=out))
    kind = _lib.BEAM_OUT_FP32 if out_dtype is torch.float32 else _lib.BEAM_OUT_BF16
    lib, s = _lib.load(), _raw_stream(stream, a)
    if grouped:
        st = lib.beam_matmul_fp8_experts(s, a.data_ptr(), a_scale.data_ptr(), offsets.data_ptr(), w.data_ptr(),
                                         w_scale.data_ptr(), M, E, N, K, kind, out.data_ptr(), 0)
    else:
        st = lib.beam_matmul_fp8(s, a.data_ptr(), a_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(), M, N, K,
                                 kind, out.data_ptr(), 0)
    if st != 0:
        raise BeamError(st, name)
    return out


def matmul_fp8(a, a_scale, w, w_scale, out_dtype=None, out=None, stream=None):
    """Product of E4M3 tokens and channels with a scale for each block of 128.

    a: [M, K] float8_e4m3fn and a_scale: [M, ceil(K/128)] float32, as an FP8 boundary writes them;
    w: [N, K] float8_e4m3fn and w_scale: [ceil(N/128), ceil(K/128)] float32. K must be a multiple of 16.
    Returns [M, N] in out_dtype: bfloat16 (the default) or float32.
    """
    return _fp8_product(a, a_scale, None, w, w_scale, out_dtype, out, stream, "beam_matmul_fp8")


def matmul_fp8_experts(a, a_scale, offsets, w, w_scale, out_dtype=None, out=None, stream=None):
    """``matmul_fp8`` of each expert's rows with its own channels.

    a: [R, K] and a_scale, the rows sorted by expert (``moe_gather``); offsets: [E + 1] int32 as
    ``moe_sort`` gives them: expert e has the rows offsets[e] .. offsets[e + 1] - 1;
    w: [E, N, K]; w_scale: [E, ceil(N/128), ceil(K/128)]. Returns [R, N]; rows of no expert are left
    as they were (in an ``out`` that the call makes, with whatever its memory held).
    """
    if offsets is None:
        raise TypeError("offsets must be a torch.Tensor")
    return _fp8_product(a, a_scale, offsets, w, w_scale, out_dtype, out, stream, "beam_matmul_fp8_experts")


def swiglu_fp8(gate_up, offsets=None, y_fp8=None, y_scale=None, stream=None):
    """``silu(gate) * up`` of rows [gate | up], as E4M3 with one FP32 scale for each 128 values.

    gate_up: [R, 2 F] bfloat16, F a multiple of 16; offsets: int32 as ``moe_sort`` gives them: rows from
    the last one on are neither read nor written (None: all rows count).
    Returns (y_fp8 [R, F] float8_e4m3fn, y_scale [R, ceil(F/128)] float32), operands of the FP8 products.
    """
    import torch
    R, F2 = _dims(gate_up, 2)
    rows, E = (R, F2 // 2), _dims(offsets, 1)[0] if offsets is not None else 0
    ready = _ready((gate_up, torch.bfloat16, (R, F2)),
                   *(() if offsets is None else ((offsets, torch.int32, (E,)),)), *_fp8_given(y_fp8, y_scale, rows))
    if not ready:
        _check(gate_up, "gate_up", torch.bfloat16, 2)
        if offsets is not None:
            _check(offsets, "offsets", torch.int32, 1)
    if F2 % 2:
        raise ValueError("gate_up must have an even number of columns")
    if offsets is not None and E < 1:
        raise ValueError("offsets must have at least one entry")
    q, scale = _fp8_out(rows, gate_up.device, y_fp8, y_scale, stream, ready)
    if not ready:
        _on_current_device(**_given(gate_up=gate_up, offsets=offsets, y_fp8=q, y_scale=scale))
    st = _lib.load().beam_swiglu_fp8(_raw_stream(stream, gate_up), gate_up.data_ptr(),
                                     None if offsets is None else offsets.data_ptr() + 4 * (E - 1), R,
                                     _c_int(rows[1]), q.data_ptr(), scale.data_ptr())
    if st != 0:
        raise BeamError(st, "beam_swiglu_fp8")
    return q, scale


@functools.lru_cache(maxsize=4096)
def _sort_workspace(T: int, K: int, E: int) -> int:
    return max(0, _lib.load().beam_moe_sort_workspace(T, K, E))


def moe_sort(topk_idx, n_experts: int, offsets=None, slots=None, stream=None):
    """Choices sorted by expert, in their order within one.

    topk_idx: [T, topk] int32 as ``moe_route`` gives them, -1 for no expert.
    Returns (offsets int32 [n_experts + 1], slots int32 [T, topk]): expert e has the sorted rows
    offsets[e] .. offsets[e + 1] - 1; slots[t, k] is the row of choice k of token t, -1 for none.
    """
    import torch
    T, K = _dims(topk_idx, 2)
    E = _c_int(n_experts)
    ready = _ready((topk_idx, torch.int32, (T, K)),
                   *(() if offsets is None else ((offsets, torch.int32, (E + 1,)),)),
                   *(() if slots is None else ((slots, torch.int32, (T, K)),)))
    if not ready:
        _check(topk_idx, "topk_idx", torch.int32, 2)
    if E < 1:
        raise ValueError(f"n_experts must be at least 1 (got {E})")
    K = _c_int(K)
    ws_bytes = _sort_workspace(T, K, E)
    with _pool(stream):
        if offsets is None:
            offsets = torch.empty(E + 1, dtype=torch.int32, device=topk_idx.device)
        if slots is None:
            slots = torch.empty((T, K), dtype=torch.int32, device=topk_idx.device)
        ws = _workspace(ws_bytes, topk_idx.device)
    if not ready:
        _check(offsets, "offsets", torch.int32, 1)
        _check(slots, "slots", torch.int32, 2)
        _shape(offsets, "offsets", (E + 1,))
        _shape(slots, "slots", (T, K))
        _on_current_device(topk_idx=topk_idx, offsets=offsets, slots=slots)
    st = _lib.load().beam_moe_sort(_raw_stream(stream, topk_idx), topk_idx.data_ptr(), T, K, E, offsets.data_ptr(),
                                   slots.data_ptr(), ws.data_ptr() if ws_bytes else None, ws_bytes)
    if st != 0:
        raise BeamError(st, "beam_moe_sort")
    return offsets, slots


def moe_gather(x, slots, scale=None, out=None, out_scale=None, stream=None):
    """Each token's row, and its scale or row of scales, copied to the rows of its choices.

    x: [T, D] of any type whose rows are a multiple of 4 bytes; slots: [T, topk] int32 as ``moe_sort``
    gives them; scale: [T] or [T, S] float32, as a boundary writes them with y in 8 bits.
    Returns out [R, D], or (out, out_scale [R] or [R, S]) with scales; R is T * topk where the call makes them.
    Rows that no choice has are left as they were (in what the call makes: as its memory was).
    The gradient for x comes from ``moe_gather_backward``.
    """
    import torch
    T, D = _dims(x, 2)
    K = _dims(slots, 2)[1]
    S = tuple(getattr(scale, "shape", (T,)))[1:]
    if out is not None:
        R = _dims(out, 2)[0]
    else:
        R = _dims(out_scale, 1 + len(S))[0] if out_scale is not None else T * K
    dtype = getattr(x, "dtype", None)
    ready = _ready((x, dtype, (T, D)), (slots, torch.int32, (T, K)),
                   *(() if scale is None else ((scale, torch.float32, (T, *S)),)),
                   *(() if out is None else ((out, dtype, (R, D)),)),
                   *(() if out_scale is None else ((out_scale, torch.float32, (R, *S)),)))
    if not ready:
        _check(x, "x", dtype, 2)
        _check(slots, "slots", torch.int32, 2)
        if slots.shape[0] != T:
            raise ValueError("shape mismatch: x [T, D]; slots [T, topk]")
        if scale is not None:
            if getattr(scale, "dim", lambda: 0)() not in (1, 2):
                raise ValueError("scale must be a 1-d or 2-d tensor")
            _check(scale, "scale", torch.float32, 1 + len(S))
            _shape(scale, "scale", (T, *S))
    if scale is None and out_scale is not None:
        raise ValueError("out_scale without scale")
    with _pool(stream):
        if out is None:
            out = torch.empty((R, D), dtype=dtype, device=x.device)
        if scale is not None and out_scale is None:
            out_scale = torch.empty((R, *S), dtype=torch.float32, device=x.device)
    if not ready:
        _check(out, "out", dtype, 2)
        _shape(out, "out", (R, D))
        if scale is not None:
            _check(out_scale, "out_scale", torch.float32, 1 + len(S))
            _shape(out_scale, "out_scale", (R, *S))
        _on_current_device(**_given(x=x, slots=slots, scale=scale, out=out, out_scale=out_scale))
    scale_bytes = 0 if scale is None else 4 * (S[0] if S else 1)
    st = _lib.load().beam_moe_gather(
        _raw_stream(stream, x), x.data_ptr(), D * x.element_size(), None if scale is None else scale.data_ptr(),
        scale_bytes, slots.data_ptr(), T, _c_int(K), R, out.data_ptr(), None if scale is None else out_scale.data_ptr())
    if st != 0:
        raise BeamError(st, "beam_moe_gather")
    return out if scale is None else (out, out_scale)


def _row_type(t, name: str) -> int:
    import torch
    dtype = getattr(t, "dtype", None)
    if dtype is torch.bfloat16:
        return _lib.BEAM_OUT_BF16
    if dtype is torch.float32:
        return _lib.BEAM_OUT_FP32
    raise TypeError(f"{name} must be a bfloat16 or float32 tensor (got {dtype})")


def _sum_rows(rows, slots, topk_w, out, stream, names, call: str):
    """``moe_combine`` and, without weights, the gradient of ``moe_gather``."""
    import torch
    kind, (R, D), (T, K) = _row_type(rows, names[0]), _dims(rows, 2), _dims(slots, 2)
    ready = _ready((rows, rows.dtype, (R, D)), (slots, torch.int32, (T, K)),
                   *(() if topk_w is None else ((topk_w, torch.float32, (T, K)),)),
                   *(() if out is None else ((out, rows.dtype, (T, D)),)))
    if not ready:
        _check(rows, names[0], rows.dtype, 2)
        _check(slots, "slots", torch.int32, 2)
        if topk_w is not None:
            _check(topk_w, "topk_w", torch.float32, 2)
            _shape(topk_w, "topk_w", (T, K))
    if out is None:
        with _pool(stream):
            out = torch.empty((T, D), dtype=rows.dtype, device=rows.device)
    if not ready:
        _check(out, names[1], rows.dtype, 2)
        _shape(out, names[1], (T, D))
        _on_current_device(**_given(**{names[0]: rows, "slots": slots, "topk_w": topk_w, names[1]: out}))
    lib, s = _lib.load(), _raw_stream(stream, rows)
    if topk_w is None:
        st = lib.beam_moe_gather_backward(s, rows.data_ptr(), slots.data_ptr(), T, _c_int(K), R, _c_int(D), kind,
                                          out.data_ptr())
    else:
        st = lib.beam_moe_combine(s, rows.data_ptr(), slots.data_ptr(), topk_w.data_ptr(), T, _c_int(K), R, _c_int(D),
                                  kind, out.data_ptr())
    if st != 0:
        raise BeamError(st, call)
    return out


def moe_gather_backward(drows, slots, dx=None, stream=None):
    """Gradient of ``moe_gather`` for x: dx[t] = sum over k of drows[slots[t, k]].

    drows: [R, D] bfloat16 or float32, D a multiple of 8; slots: [T, topk] int32. FP32 sums in the order
    of the choices, rounded once. Returns dx [T, D] of drows' type (0 for a token without choices).
    """
    return _sum_rows(drows, slots, None, dx, stream, ("drows", "dx"), "beam_moe_gather_backward")


def moe_combine(rows, slots, topk_w, out=None, stream=None):
    """The experts' outputs back to their tokens: out[t] = sum over k of topk_w[t, k] rows[slots[t, k]].

    rows: [R, D] bfloat16 or float32, D a multiple of 8; slots: [T, topk] int32 as ``moe_sort`` gives
    them; topk_w: [T, topk] float32. FP32 multiply-adds in the order of the choices, rounded once, as
    ``moe_combine_boundary`` makes its x: ``boundary_fused`` on the result gives the same bits.
    Returns out [T, D] of the rows' type (0 for a token without choices). Gradients come from
    ``moe_combine_backward``.
    """
    if topk_w is None:
        raise TypeError("topk_w must be a torch.Tensor")
    return _sum_rows(rows, slots, topk_w, out, stream, ("rows", "out"), "beam_moe_combine")


def moe_combine_backward(dx, rows, slots, topk_w, drows=None, dw=None, stream=None):
    """Gradients of ``moe_combine`` for the gradient dx [T, D] of its result.

    Returns (drows [R, D] of the rows' type: topk_w[t, k] dx[t] at slots[t, k], rows that no choice has
    left as they were; dw float32 [T, topk]: the product of dx[t] with the choice's row, 0 for none).
    """
    import torch
    kind, (R, D), (T, K) = _row_type(rows, "rows"), _dims(rows, 2), _dims(slots, 2)
    dtype = rows.dtype
    ready = _ready((dx, dtype, (T, D)), (rows, dtype, (R, D)), (slots, torch.int32, (T, K)),
                   (topk_w, torch.float32, (T, K)), *(() if drows is None else ((drows, dtype, (R, D)),)),
                   *(() if dw is None else ((dw, torch.float32, (T, K)),)))
    if not ready:
        _check(rows, "rows", dtype, 2)
        _check(slots, "slots", torch.int32, 2)
        _check(dx, "dx", dtype, 2)
        _check(topk_w, "topk_w", torch.float32, 2)
        _shape(dx, "dx", (T, D))
        _shape(topk_w, "topk_w", (T, K))
    with _pool(stream):
        if drows is None:
            drows = torch.empty_like(rows)
        if dw is None:
            dw = torch.empty((T, K), dtype=torch.float32, device=rows.device)
    if not ready:
        _check(drows, "drows", dtype, 2)
        _check(dw, "dw", torch.float32, 2)
        _shape(drows, "drows", (R, D))
        _shape(dw, "dw", (T, K))
        _on_current_device(dx=dx, rows=rows, slots=slots, topk_w=topk_w, drows=drows, dw=dw)
    st = _lib.load().beam_moe_combine_backward(
        _raw_stream(stream, rows), dx.data_ptr(), rows.data_ptr(), slots.data_ptr(), topk_w.data_ptr(), T, _c_int(K), R,
        _c_int(D), kind, drows.data_ptr(), dw.data_ptr())
    if st != 0:
        raise BeamError(st, "beam_moe_combine_backward")
    return drows, dw


def moe_route(logits, bias, n_group: int = 8, topk_group: int = 4, topk: int = 8,
              route_scale: float = 2.5, idx=None, w=None, stream=None, pdl: bool = False):
    """Group-limited top-k routing on torch CUDA tensors.

    logits: [T, 256] float32 router logits; bias: [256] float32 correction bias.
    pdl: launch with programmatic dependent launch (BEAM_OPT_PDL).
    Returns (idx int32 [T, topk], w float32 [T, topk]).
    """
    import torch
    _check(logits, "logits", torch.float32, 2)
    _check(bias, "bias", torch.float32, 1)
    T, E = logits.shape
    if bias.shape[0] != E:
        raise ValueError("bias must have one entry per expert")
    with _pool(stream):
        if idx is None:
            idx = torch.empty((T, topk), dtype=torch.int32, device=logits.device)
        if w is None:
            w = torch.empty((T, topk), dtype=torch.float32, device=logits.device)
    _check(idx, "idx", torch.int32, 2)
    _check(w, "w", torch.float32, 2)
    _shape(idx, "idx", (T, topk))
    _shape(w, "w", (T, topk))
    _on_current_device(logits=logits, bias=bias, idx=idx, w=w)
    st = _lib.load().beam_moe_route_ex(_stream_ptr(stream), logits.data_ptr(), bias.data_ptr(), T, _c_int(E),
                                       _c_int(n_group), _c_int(topk_group), _c_int(topk), float(route_scale),
                                       idx.data_ptr(), w.data_ptr(), _lib.BEAM_OPT_PDL if pdl else 0)
    if st != 0:
        raise BeamError(st, "beam_moe_route_ex")
    return idx, w


def _sequences(seq_offsets) -> int:
    """S, of [S + 1] sequence offsets (1 for None)."""
    import torch
    if seq_offsets is None:
        return 1
    _check(seq_offsets, "seq_offsets", torch.int32, 1)
    if seq_offsets.shape[0] < 2:
        raise ValueError("seq_offsets must have at least two entries")
    return seq_offsets.shape[0] - 1


def _given(**operands) -> dict:
    return {name: t for name, t in operands.items() if t is not None}


@functools.lru_cache(maxsize=4096)
def _balance_workspace(T: int, E: int, S: int) -> int:
    return max(0, _lib.load().beam_moe_balance_workspace(T, E, S))


def moe_balance_loss(logits, topk_idx, alpha: float, seq_offsets=None, loss=None, counts=None,
                     stream=None):
    """Sequence-wise balance loss of the router, with the per-expert counts.

    logits: [T, E] float32; topk_idx: [T, topk] int32, as ``moe_route`` gives them;
    seq_offsets: [S + 1] int32 first tokens of the sequences and the end of the last (None: one
    sequence); tokens outside are padding and count for nothing.
    Returns (loss float32 [S], counts int32 [S, E]). Autograd does not see the call: the gradient
    for the logits comes from ``moe_balance_loss_backward``.
    """
    import torch
    S = _sequences(seq_offsets)
    (T, E), (_, K) = _dims(logits, 2), _dims(topk_idx, 2)
    ready = _ready((logits, torch.float32, (T, E)), (topk_idx, torch.int32, (T, K)),
                   *(() if seq_offsets is None else ((seq_offsets, torch.int32, (S + 1,)),)),
                   *(() if loss is None else ((loss, torch.float32, (S,)),)),
                   *(() if counts is None else ((counts, torch.int32, (S, E)),)))
    if not ready:
        _check(logits, "logits", torch.float32, 2)
        _check(topk_idx, "topk_idx", torch.int32, 2)
        if topk_idx.shape[0] != T:
            raise ValueError("shape mismatch: logits [T, E]; topk_idx [T, topk]")
    E, K = _c_int(E), _c_int(K)
    ws_bytes = _balance_workspace(T, E, S)
    with _pool(stream):
        if loss is None:
            loss = torch.empty(S, dtype=torch.float32, device=logits.device)
        if counts is None:
            counts = torch.empty((S, E), dtype=torch.int32, device=logits.device)
        ws = _workspace(ws_bytes, logits.device)
    if not ready:
        _check(loss, "loss", torch.float32, 1)
        _check(counts, "counts", torch.int32, 2)
        _shape(loss, "loss", (S,))
        _shape(counts, "counts", (S, E))
        _on_current_device(**_given(logits=logits, topk_idx=topk_idx, seq_offsets=seq_offsets, loss=loss,
                                    counts=counts))
    st = _lib.load().beam_moe_balance_loss(
        _raw_stream(stream, logits), logits.data_ptr(), topk_idx.data_ptr(),
        None if seq_offsets is None else seq_offsets.data_ptr(), T, E, K, S, float(alpha), loss.data_ptr(),
        counts.data_ptr(), ws.data_ptr() if ws_bytes else None, ws_bytes)
    if st != 0:
        raise BeamError(st, "beam_moe_balance_loss")
    return loss, counts


def moe_balance_loss_backward(dloss, logits, counts, topk: int, alpha: float, seq_offsets=None,
                              dlogits=None, stream=None):
    """Gradient of ``(dloss * loss).sum()`` for the logits of ``moe_balance_loss``.

    dloss: [S] float32; counts: [S, E] int32 as ``moe_balance_loss`` returned them; the other
    arguments as there. Returns dlogits float32 [T, E] (0 for padding).
    """
    import torch
    S = _sequences(seq_offsets)
    T, E = rows = _dims(logits, 2)
    ready = _ready((dloss, torch.float32, (S,)), (logits, torch.float32, rows), (counts, torch.int32, (S, E)),
                   *(() if seq_offsets is None else ((seq_offsets, torch.int32, (S + 1,)),)),
                   *(() if dlogits is None else ((dlogits, torch.float32, rows),)))
    if not ready:
        _check(dloss, "dloss", torch.float32, 1)
        _check(logits, "logits", torch.float32, 2)
        _check(counts, "counts", torch.int32, 2)
        _shape(dloss, "dloss", (S,))
        _shape(counts, "counts", (S, E))
    if dlogits is None:
        with _pool(stream):
            dlogits = torch.empty_like(logits)
    if not ready:
        _check(dlogits, "dlogits", torch.float32, 2)
        _shape(dlogits, "dlogits", (T, E))
        _on_current_device(**_given(dloss=dloss, logits=logits, counts=counts, seq_offsets=seq_offsets,
                                    dlogits=dlogits))
    st = _lib.load().beam_moe_balance_loss_backward(
        _raw_stream(stream, logits), dloss.data_ptr(), logits.data_ptr(), counts.data_ptr(),
        None if seq_offsets is None else seq_offsets.data_ptr(), T, _c_int(E), _c_int(topk), S, float(alpha),
        dlogits.data_ptr())
    if st != 0:
        raise BeamError(st, "beam_moe_balance_loss_backward")
    return dlogits


def router_sigmoid(z, out=None, stream=None, fast: bool = False):
    """The router's correctly rounded FP32 sigmoid of every element of ``z`` (float32 CUDA
    tensor, any shape, contiguous); ``out`` may be ``z`` (in place). With ``fast``, the
    routing first pass's approximation instead (within 2^-19 of the exact sigmoid)."""
    import torch
    if not isinstance(z, torch.Tensor) or z.dtype != torch.float32 or not z.is_contiguous():
        raise TypeError("z must be a contiguous float32 tensor")
    if out is None:
        with _pool(stream):
            out = torch.empty_like(z)
    if not isinstance(out, torch.Tensor) or out.dtype != torch.float32 or not out.is_contiguous():
        raise TypeError("out must be a contiguous float32 tensor")
    _shape(out, "out", tuple(z.shape))
    _on_current_device(z=z, out=out)
    fn = _lib.load().beam_router_sigmoid_fast if fast else _lib.load().beam_router_sigmoid
    st = fn(_stream_ptr(stream), z.data_ptr(), out.data_ptr(), z.numel())
    if st != 0:
        raise BeamError(st, "beam_router_sigmoid_fast" if fast else "beam_router_sigmoid")
    return out


def qk_norm(q, k, q_w, k_w, pos, eps: float = 1e-6, mode: str = "rope", rope_table=None,
            stream=None, force_exact: bool = False, pdl: bool = False):
    """Per-head Q/K RMSNorm then RoPE (mode "rope") or SSMax (mode "ssmax"), in place.

    q: [T, n_q, 128] bf16; k: [T, n_kv, 128] bf16; q_w, k_w: [128] bf16; pos: [T] int32;
    rope_table: [max_pos, 128] float32 (cos | sin), needed for mode "rope".
    """
    import torch
    _check(q, "q", torch.bfloat16, 3)
    _check(k, "k", torch.bfloat16, 3)
    _check(q_w, "q_w", torch.bfloat16, 1)
    _check(k_w, "k_w", torch.bfloat16, 1)
    _check(pos, "pos", torch.int32, 1)
    T = q.shape[0]
    if k.shape[0] != T or pos.shape[0] != T or q.shape[2] != k.shape[2]:
        raise ValueError("shape mismatch: q [T, nq, 128], k [T, nk, 128], pos [T]")
    hd = q.shape[2]
    _shape(q_w, "q_w", (hd,))
    _shape(k_w, "k_w", (hd,))
    m = {"rope": _lib.BEAM_QK_ROPE, "ssmax": _lib.BEAM_QK_SSMAX}[mode]
    tab, max_pos = 0, 0
    ops = dict(q=q, k=k, q_w=q_w, k_w=k_w, pos=pos)
    if mode == "rope":
        _check(rope_table, "rope_table", torch.float32, 2)
        if rope_table.shape[1] != hd:
            raise ValueError(f"rope_table must be [max_pos, {hd}] (cos | sin)")
        tab, max_pos = rope_table.data_ptr(), rope_table.shape[0]
        ops["rope_table"] = rope_table
    _on_current_device(**ops)
    st = _lib.load().beam_qk_norm_ex(_stream_ptr(stream), q.data_ptr(), k.data_ptr(), q_w.data_ptr(),
                                     k_w.data_ptr(), pos.data_ptr(), tab or None, max_pos, T,
                                     _c_int(q.shape[1]), _c_int(k.shape[1]), _c_int(q.shape[2]), float(eps), m,
                                     (_lib.BEAM_OPT_FORCE_EXACT_SUM if force_exact else 0)
                                     | (_lib.BEAM_OPT_PDL if pdl else 0))
    if st != 0:
        raise BeamError(st, "beam_qk_norm")
    return q, k


def sync_status(stream=None) -> None:
    """Synchronise the stream and raise BeamError if a kernel reported a device-side error."""
    st = _lib.load().beam_sync_status(_stream_ptr(stream))
    if st != 0:
        raise BeamError(st, "beam_sync_status")


def exact_sum_count(reset: bool = False, stream=None) -> int:
    """Row sums that took the exact integer path on this device (diagnostics)."""
    v = ctypes.c_uint64(0)
    st = _lib.load().beam_exact_sum_count(_stream_ptr(stream), ctypes.byref(v), int(reset))
    if st != 0:
        raise BeamError(st, "beam_exact_sum_count")
    return int(v.value)


def version() -> int:
    return int(_lib.load().beam_version())
