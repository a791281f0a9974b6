"""What writes the FP8 products' operands, on the GPU: the boundaries with y as FP8 (bit for bit against the oracle's
BF16 boundary and the formula) and the experts' activation (against 64 bits)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import sandwich_norm_residual_gb300 as snr
from sandwich_norm_residual_gb300 import _lib, build

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    oracle.build()
    snr.library()


def e4m3(v: np.ndarray) -> np.ndarray:
    """FP32 -> the nearest E4M3 number (ties to even), largest 448, by its definition in 64 bits."""
    v = v.astype(np.float64)
    _, e = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(e, -5) - 4)
    return np.clip(np.rint(v / step) * step, -448, 448)


def quantised(y: np.ndarray):
    """(values of the codes, scales) of FP32 rows by the header's formula."""
    T, D = y.shape
    B = -(-D // 128)
    v = np.zeros((T, B * 128), np.float32)
    v[:, :D] = y
    v = v.reshape(T, B, 128)
    with np.errstate(all="ignore"):
        amax = np.abs(v).max(2)  # a NaN stays
        scale = amax / np.float32(448)
        up = np.where(amax < np.float32(2.0 ** -100), np.float32(2.0 ** 64), np.float32(1))
        inv = np.float32(448) / (amax * up)
        q = e4m3((v * up[:, :, None]) * inv[:, :, None])
    q[~((amax > 0) & np.isfinite(amax))] = 0
    return q.reshape(T, B * 128)[:, :D], scale


def check(q, s, y):
    ref, scale = quantised(y)
    assert np.array_equal(s.cpu().numpy(), scale, equal_nan=True)
    got = q.float().cpu().numpy()
    assert np.array_equal(got, ref)
    assert np.array_equal(np.signbit(got), np.signbit(ref) | (np.signbit(y) & (got == 0) & (ref == 0) & np.signbit(got)))


def u16(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


def f32(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32)


def bf(rng, *s, scale=1.0):
    return torch.from_numpy((rng.standard_normal(s) * scale).astype(np.float32)).to(torch.bfloat16)


@pytest.mark.parametrize("T,D,n", [(1, 8, 1), (3, 120, 2), (5, 128, 7), (4, 136, 3), (2, 5120, 20), (130, 5120, 104),
                                   (17, 4104, 50), (9, 1000, 5), (3, 32768, 9), (300, 2568, 12), (2000, 640, 6)])
def test_dense(T, D, n):
    rng = np.random.default_rng(T + D)
    h, x, pw, qw = bf(rng, T, D), bf(rng, T, D, scale=3), bf(rng, D), bf(rng, D)
    hd = h.cuda()
    q, s = snr.boundary_fused_fp8(hd, x.cuda(), pw.cuda(), qw.cuda(), n)
    snr.sync_status()
    href, yref = oracle.boundary(h, x, pw, qw, n, 1e-6)
    assert q.dtype == FP8 and q.shape == (T, D) and s.shape == (T, -(-D // 128))
    assert np.array_equal(u16(hd), href)
    check(q, s, f32(yref))


@pytest.mark.parametrize("scale", [1.0, 2.5])
@pytest.mark.parametrize("T,D", [(1, 8), (5, 264), (40, 5120), (7, 4104)])
def test_moe(T, D, scale):
    rng = np.random.default_rng(T + D)
    h, e, pw, qw = bf(rng, T, D), bf(rng, T, 8, D), bf(rng, D), bf(rng, D)
    w = torch.from_numpy(rng.random((T, 8)).astype(np.float32))
    hd, h2 = h.cuda(), h.cuda()
    q, s = snr.moe_combine_boundary_fp8(hd, e.cuda(), w.cuda(), pw.cuda(), qw.cuda(), 20, route_scale=scale)
    y = snr.moe_combine_boundary(h2, e.cuda(), w.cuda(), pw.cuda(), qw.cuda(), 20, route_scale=scale)
    snr.sync_status()
    assert torch.equal(hd, h2)
    check(q, s, y.float().cpu().numpy())
    if scale == 1.0:
        href, yref = oracle.moe_boundary(h, e, w, pw, qw, 20, 1e-6)
        assert np.array_equal(u16(hd), href) and np.array_equal(u16(y), yref)


@pytest.mark.parametrize("vec", range(1, 9))
@pytest.mark.parametrize("exact", [False, True])
def test_every_launch_shape_gives_the_same(vec, exact):
    rng = np.random.default_rng(1)
    for D in (1024, 1288, 2560):
        T = 30
        h, x, pw, qw = (t.cuda() for t in (bf(rng, T, D), bf(rng, T, D), bf(rng, D), bf(rng, D)))
        h0 = h.clone()
        q0, s0 = snr.boundary_fused_fp8(h0, x, pw, qw, 5)
        opts = dict(vec_per_thread=vec, ctas_per_sm=1 + vec % 3, flags=_lib.BEAM_OPT_FORCE_EXACT_SUM if exact else 0)
        q, s = snr.boundary_fused_fp8(h, x, pw, qw, 5, opts=opts)
        snr.sync_status()
        assert torch.equal(q.view(torch.uint8), q0.view(torch.uint8)) and torch.equal(s, s0) and torch.equal(h, h0)


def test_tiny_zero_and_non_finite_blocks():
    """Pre-norm weights make blocks of y tiny, zero, infinite or NaN; the others stay as they are."""
    T, D = 6, 1024
    rng = np.random.default_rng(2)
    h, x, pw, qw = bf(rng, T, D), bf(rng, T, D), bf(rng, D), bf(rng, D)
    qw[128:256] = 0
    qw[256:384] *= 2.0 ** -110
    qw[384:512] *= 2.0 ** -125
    qw[512] = float("inf")
    qw[640 + 5] = float("nan")
    qw[768:896] *= 2.0 ** 100
    hd = h.cuda()
    q, s = snr.boundary_fused_fp8(hd, x.cuda(), pw.cuda(), qw.cuda(), 3)
    snr.sync_status()
    _, yref = oracle.boundary(h, x, pw, qw, 3, 1e-6)
    check(q, s, f32(yref))
    sn = s.cpu().numpy()
    assert (sn[:, 1] == 0).all() and np.isinf(sn[:, 4]).all() and np.isnan(sn[:, 5]).all()
    assert not q.view(torch.uint8)[:, 512:768].any()


def test_pdl_chain_in_a_graph():
    rng = np.random.default_rng(3)
    T, D = 64, 5120
    h, pw, qw = bf(rng, T, D).cuda(), bf(rng, D).cuda(), bf(rng, D).cuda()
    xs = [bf(rng, T, D).cuda() for _ in range(5)]
    h0 = h.clone()
    want = [snr.boundary_fused_fp8(h0, x, pw, qw, 2 + i) for i, x in enumerate(xs)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = [snr.boundary_fused_fp8(h, x, pw, qw, 2 + i, opts=dict(flags=_lib.BEAM_OPT_PDL)) for i, x in enumerate(xs)]
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, h0)
    for (q, s), (q0, s0) in zip(got, want):
        assert torch.equal(q.view(torch.uint8), q0.view(torch.uint8)) and torch.equal(s, s0)


# ---------------------------------------------------------------- the activation

def check_swiglu(x, q, s):
    """y's error, relative: (6 + 2 |g|) 2^-24 by the header. The scale then has that of the block's largest y and half a
    step (2^-24); a value is off by half a step of E4M3 (2^-4 of it, 2^-10 below 2^-6) and by what its scaling
    moved it: the errors of y, of the largest and four roundings."""
    F = x.shape[1] // 2
    g, u = x[:, :F].double(), x[:, F:].double()
    y = g * torch.sigmoid(g) * u
    err = (6 + 2 * g.abs()) * 2.0 ** -24 * y.abs() + 1e-43
    pad = lambda t: torch.nn.functional.pad(t, (0, -F % 128)).view(len(t), -1, 128)  # noqa: E731
    top = pad(y.abs()).amax(2)
    top_err = pad(err).amax(2)
    sd = s.double()
    assert ((sd - top / 448).abs() <= top_err / 448 + 2.0 ** -24 * sd).all()
    value = pad(q.double()) * sd[:, :, None]
    code = pad(y) / torch.where(sd > 0, sd, 1.0)[:, :, None]
    half = torch.maximum(2.0 ** -4 * code.abs(), torch.full_like(code, 2.0 ** -10)) * sd[:, :, None]
    rel = (top_err / top.clamp(min=1e-300) + 4 * 2.0 ** -24)[:, :, None]
    assert ((value - pad(y)).abs() <= half * (1 + 2.0 ** -10) + 2 * pad(err) + 2 * rel * pad(y).abs()).all()


@pytest.mark.parametrize("R,F", [(1, 16), (1, 2560), (3, 128), (7, 144), (512, 2560), (33, 240), (1000, 272), (5000, 1040), (9, 65536)])
def test_swiglu(R, F):
    g = torch.Generator(device="cuda")
    g.manual_seed(R + F)
    x = (torch.randn(R, 2 * F, device="cuda", generator=g) * 4).to(torch.bfloat16)
    q, s = snr.swiglu_fp8(x)
    snr.sync_status()
    assert q.dtype == FP8 and q.shape == (R, F) and s.shape == (R, -(-F // 128))
    check_swiglu(x, q, s)


def test_swiglu_of_large_small_and_zero_gates():
    F = 256
    x = torch.zeros(8, 2 * F)
    x[0, :F], x[0, F:] = -200.0, 3.0    # e^-g overflows: 0
    x[1, :F], x[1, F:] = 200.0, -3.0    # the gate itself
    x[2, :F], x[2, F:] = 1e-30, 1e-8    # below 2^-100: brought up first
    x[3, 1], x[3, F + 1] = 5.0, 2.0     # a block with one value
    x[4, :F], x[4, F:] = -30.0, 1.0
    x[6, 3], x[6, F + 3] = float("inf"), 1.0
    x[7, 130], x[7, F + 130] = 1.0, float("nan")
    x = x.to(torch.bfloat16).cuda()
    q, s = snr.swiglu_fp8(x)
    snr.sync_status()
    check_swiglu(x[:6], q.view(torch.uint8)[:6].view(FP8), s[:6])
    assert not s[0].any() and not q.view(torch.uint8)[0].bitwise_and(127).any()
    assert s[6, 0].isinf() and s[7, 1].isnan() and not q.view(torch.uint8)[6:].bitwise_and(127).any()
    assert s[6, 1] == 0 and s[7, 0] == 0


@pytest.mark.parametrize("live", [0, 1, 37, 300])
def test_swiglu_leaves_rows_behind_the_last_expert(live):
    R, F = 300, 400
    x = torch.randn(R, 2 * F, device="cuda").to(torch.bfloat16)
    x[live:] = float("nan")
    off = torch.tensor([0, live // 2, live], dtype=torch.int32, device="cuda")
    q = torch.full((R, F), 3, dtype=torch.uint8, device="cuda").view(FP8)
    s = torch.full((R, 4), -1.0, device="cuda")
    snr.swiglu_fp8(x, offsets=off, y_fp8=q, y_scale=s)
    snr.sync_status()
    assert (q.view(torch.uint8)[live:] == 3).all() and (s[live:] == -1).all()
    if live:
        check_swiglu(x[:live], q.view(torch.uint8)[:live].view(FP8), s[:live])


@pytest.mark.parametrize("count", [-1, 301, 2 ** 31 - 1, -2 ** 31])
def test_swiglu_with_a_bad_count_is_reported(count):
    x = torch.randn(300, 64, device="cuda").to(torch.bfloat16)
    buf = torch.full((320, 32), 3, dtype=torch.uint8, device="cuda")
    q = buf[10:310].view(FP8)
    snr.swiglu_fp8(x, offsets=torch.tensor([count], dtype=torch.int32, device="cuda"), y_fp8=q)
    with pytest.raises(snr.BeamError) as e:
        snr.sync_status()
    assert e.value.status == _lib.BEAM_ERR_ARG
    assert (buf[:10] == 3).all() and (buf[310:] == 3).all()


@pytest.mark.slow
def test_swiglu_past_32_bits():
    R, F = 70000, 16384
    x = torch.zeros(R, 2 * F, dtype=torch.bfloat16, device="cuda")  # 4.6 GB
    x[-1], x[R // 2] = 2.0, 3.0
    q, s = snr.swiglu_fp8(x)
    snr.sync_status()
    for r in (0, R // 2, R - 1):
        check_swiglu(x[r:r + 1], q.view(torch.uint8)[r:r + 1].view(FP8), s[r:r + 1])
    assert int((s != 0).any(1).sum()) == 2
