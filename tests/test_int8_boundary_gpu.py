"""GPU parity of the boundaries whose y leaves as int8: h', codes and scales bit for bit against
the CPU oracle's BF16 boundary followed by the documented quantisation, written out in numpy."""
from __future__ import annotations

import os

import numpy as np
import pytest
import torch

import oracle
import sandwich_norm_residual_gb300 as snr
import synth
from parity import bits
from sandwich_norm_residual_gb300 import _lib, build
from synth import DENSE_PREFILL_T16384, MOE_T16384

pytestmark = pytest.mark.gpu
THREADS = max(1, min(32, os.cpu_count() or 1))


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    snr.library()


def quantise(y_u16):
    """[T, D] BF16 bits -> int8 codes and FP32 scales, by the header's formula."""
    y = (y_u16.astype(np.uint32) << 16).view(np.float32)
    a = np.abs(y).max(1)  # NaN when the row holds one
    with np.errstate(all="ignore"):
        scale = a / np.float32(127)
        up = np.where(a < np.float32(2.0) ** -100, np.float32(2.0) ** 64, np.float32(1)).astype(np.float32)
        inv = np.float32(127) / (a * up)
        live = (a > 0) & np.isfinite(a)
        q = np.rint((y * up[:, None]) * inv[:, None])
    return np.where(live[:, None], q, 0).astype(np.int8), scale


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def random_inputs(T, D, seed, moe=False):
    rng = np.random.default_rng(seed)
    d = dict(h=bf16(rng.standard_normal((T, D))), post_w=bf16(1 + 0.1 * rng.standard_normal(D)),
             pre_w=bf16(1 + 0.1 * rng.standard_normal(D)))
    if moe:
        d["expert_out"] = bf16(rng.standard_normal((T, 8, D)))
        d["topk_w"] = torch.from_numpy(rng.random((T, 8)).astype(np.float32))
    else:
        d["x"] = bf16(rng.standard_normal((T, D)))
    return d


def run(inp, n, eps, stream=None, **kw):
    d = {k: v.cuda() for k, v in inp.items()}
    if "x" in d:
        q, s = snr.boundary_fused_int8(d["h"], d["x"], d["post_w"], d["pre_w"], n, eps, stream=stream, **kw)
    else:
        q, s = snr.moe_combine_boundary_int8(d["h"], d["expert_out"], d["topk_w"], d["post_w"], d["pre_w"], n,
                                             eps, stream=stream, **kw)
    snr.sync_status(stream)
    return bits(d["h"]), q.cpu().numpy(), s.cpu().numpy()


def want(inp, n, eps):
    if "x" in inp:
        h, y = oracle.boundary(inp["h"], inp["x"], inp["post_w"], inp["pre_w"], n, eps, threads=THREADS)
    else:
        h, y = oracle.moe_boundary(inp["h"], inp["expert_out"], inp["topk_w"], inp["post_w"], inp["pre_w"], n,
                                   eps, threads=THREADS)
    return (h, *quantise(y))


def same(got, ref):
    assert np.array_equal(got[0], ref[0])
    assert np.array_equal(got[1], ref[1])
    assert np.array_equal(got[2], ref[2], equal_nan=True)


SHAPES = [(1, 8, 2), (3, 16, 1), (5, 264, 3), (1, 5120, 2), (67, 5120, 104), (9, 4104, 7), (4, 8192, 105),
          (2, 32768, 5), (700, 40, 9)]


@pytest.mark.parametrize("moe", [False, True])
@pytest.mark.parametrize("T,D,n", SHAPES)
def test_shapes(T, D, n, moe):
    inp = random_inputs(T, D, T * 131 + D, moe)
    same(run(inp, n, 1e-6), want(inp, n, 1e-6))


@pytest.mark.parametrize("moe", [False, True])
def test_prefill_workload(moe):
    cfg = MOE_T16384 if moe else DENSE_PREFILL_T16384
    inp = synth.moe_inputs(cfg, rows=2048) if moe else synth.dense_inputs(cfg, rows=4096)
    same(run(inp, cfg.n, cfg.eps), want(inp, cfg.n, cfg.eps))


@pytest.mark.parametrize("moe", [False, True])
def test_every_launch_shape_forced_exact_sums_and_pdl(moe):
    inp = random_inputs(33, 1280, 5, moe)
    ref = want(inp, 6, 1e-6)
    for v in range(1, 9):
        same(run(inp, 6, 1e-6, opts=dict(vec_per_thread=v)), ref)
    for o in (dict(ctas_per_sm=1), dict(prefetch_rows=-1), dict(prefetch_rows=3),
              dict(flags=_lib.BEAM_OPT_FORCE_EXACT_SUM), dict(flags=_lib.BEAM_OPT_PDL)):
        same(run(inp, 6, 1e-6, opts=o), ref)


@pytest.mark.parametrize("moe", [False, True])
def test_zero_tiny_and_non_finite_rows(moe):
    T, D = 8, 512
    inp = random_inputs(T, D, 11, moe)
    branch = inp["expert_out"][:, 0] if moe else inp["x"]
    inp["h"][1] = 0                      # n = 1 below: h' is the normalised branch alone
    branch[2, 5] = float("nan")
    branch[3, 7] = float("inf")
    branch[4, :] = 0
    if moe:
        inp["expert_out"][4] = 0
        inp["topk_w"][5] = float("nan")
    # weights that make every y tiny: below 2^-100, down to BF16's subnormals
    for scale in (1.0, 2.0 ** -110, 2.0 ** -132):
        inp["pre_w"] = bf16(np.full(D, scale))
        inp["pre_w"][::3] = 0
        ref = want(inp, 1, 1e-6)
        same(run(inp, 1, 1e-6), ref)
        assert not np.isfinite(ref[2][2]) and not ref[1][2].any()
        assert ref[2][4] == 0 and not ref[1][4].any()


def test_codes_reach_both_ends_and_stand_for_y_within_half_a_step():
    inp = random_inputs(257, 1032, 3)
    h, q, s = run(inp, 4, 1e-6)
    _, y = oracle.boundary(inp["h"], inp["x"], inp["post_w"], inp["pre_w"], 4, 1e-6)
    yf = (y.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    assert q.max() == 127 and q.min() == -127 and (np.abs(q.astype(int)).max(1) == 127).all()
    # half a step, and the FP32 roundings of 127/amax, the product and amax/127 (3 half-ulps on up to 127 steps)
    assert (np.abs(q * s[:, None].astype(np.float64) - yf) <= s[:, None] * (0.5 + 127 * 3 * 2.0 ** -24)).all()


def test_route_scale_matches_the_scaled_bf16_combine():
    inp = random_inputs(19, 648, 8, moe=True)
    d = {k: v.cuda() for k, v in inp.items()}
    h2 = d["h"].clone()
    y = snr.moe_combine_boundary(h2, d["expert_out"], d["topk_w"], d["post_w"], d["pre_w"], 3, 1e-6,
                                 route_scale=2.5)
    got = run(inp, 3, 1e-6, route_scale=2.5)
    same(got, (bits(h2), *quantise(bits(y))))


def test_branch_may_be_the_stream_and_neighbours_stay():
    T, D = 5, 264
    inp = random_inputs(T, D, 21)
    inp["x"] = inp["h"].clone()
    h, y = oracle.boundary(inp["h"], inp["x"], inp["post_w"], inp["pre_w"], 3, 1e-6)
    g = inp["h"].cuda()
    codes = torch.full((T + 2, D), 77, dtype=torch.int8, device="cuda")
    scales = torch.full((T + 8,), 77.0, device="cuda")
    pad = 16  # bytes: keeps the operands 16-byte aligned and the guard directly beside them
    q = codes.view(-1)[pad:pad + T * D].view(T, D)
    s = scales[4:4 + T]
    snr.boundary_fused_int8(g, g, inp["post_w"].cuda(), inp["pre_w"].cuda(), 3, 1e-6, y_int8=q, y_scale=s)
    snr.sync_status()
    same((bits(g), q.cpu().numpy(), s.cpu().numpy()), (h, *quantise(y)))
    flat = codes.view(-1)
    assert (flat[:pad] == 77).all() and (flat[pad + T * D:] == 77).all()
    assert (scales[:4] == 77).all() and (scales[4 + T:] == 77).all()


def test_no_tokens_and_a_side_stream():
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    q, s = snr.boundary_fused_int8(e, e, w, w, 2)
    assert q.shape == (0, 64) and s.shape == (0,)
    inp = random_inputs(40, 520, 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    same(run(inp, 2, 1e-6, stream=side), want(inp, 2, 1e-6))


@pytest.mark.slow
def test_rows_past_32_bits():
    T, D = 420_000, 5120  # 2.15e9 elements
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    h = torch.randn((T, D), dtype=torch.bfloat16, device="cuda")
    x = torch.randn((T, D), dtype=torch.bfloat16, device="cuda")
    tail = slice(T - 100, T)
    inp = dict(h=h[tail].cpu(), x=x[tail].cpu(), post_w=w.cpu(), pre_w=w.cpu())
    q, s = snr.boundary_fused_int8(h, x, w, w, 9)
    snr.sync_status()
    same((bits(h[tail]), q[tail].cpu().numpy(), s[tail].cpu().numpy()), want(inp, 9, 1e-6))
