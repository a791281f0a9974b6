"""Bytes that the FP8 boundaries and the activation write: signs of values that round to zero are kept, blocks of zeros and
blocks that hold an infinity or a NaN are bytes of 0."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import sandwich_norm_residual_gb300 as snr
from sandwich_norm_residual_gb300 import build
from test_fp8_rows_gpu import FP8, bf, f32, quantised

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    oracle.build()
    snr.library()


def same_bytes(q, y):
    """The codes are those of the header's formula, bit for bit, negative zeros among them."""
    ref = quantised(y)[0]
    want = torch.from_numpy(ref).to(torch.float32).to(FP8).view(torch.uint8).numpy()
    assert np.array_equal(np.signbit(ref), want >= 0x80)
    assert np.array_equal(q.view(torch.uint8).cpu().numpy(), want)
    return want


def inputs(T, D):
    rng = np.random.default_rng(T + D)
    h, x, pw, qw = bf(rng, T, D), bf(rng, T, D), bf(rng, D), bf(rng, D)
    qw[64:120] *= 2.0 ** -14       # beside larger ones of their block: round to a zero of their sign
    qw[128:256] = 0
    qw[256:384] = -0.0
    qw[384:512] *= 2.0 ** -110     # brought up first
    qw[512] = float("inf")
    qw[640 + 5] = float("nan")
    qw[768:800] = float("-inf")
    return h, x, pw, qw


@pytest.mark.parametrize("T,D", [(6, 1024), (40, 904), (3, 5120)])
def test_dense(T, D):
    h, x, pw, qw = inputs(T, D)
    hd = h.cuda()
    q, s = snr.boundary_fused_fp8(hd, x.cuda(), pw.cuda(), qw.cuda(), 3)
    snr.sync_status()
    y = f32(oracle.boundary(h, x, pw, qw, 3, 1e-6)[1])
    want = same_bytes(q, y)
    assert (want == 0x80).any()
    raw = q.view(torch.uint8)
    assert np.signbit(y[:, 128:384]).any()  # zeros of both signs went in
    for block in (1, 2, 4, 5, 6):
        assert not raw[:, 128 * block:128 * block + 128].any()
    sn = s.cpu().numpy()
    assert (sn[:, 1:3] == 0).all() and not np.signbit(sn[:, 1:3]).any()
    # 40 by 904: h' is 0 once where the weight is -inf, 0 * -inf is NaN and the block's scale with it
    assert np.array_equal(sn, quantised(y)[1], equal_nan=True)
    assert np.isposinf(sn[:, [4, 6]]).mean() > 0.98 and not np.isfinite(sn[:, 4:7]).any() and np.isnan(sn[:, 5]).all()


def test_moe():
    T, D = 5, 1024
    h, _, pw, qw = inputs(T, D)
    rng = np.random.default_rng(7)
    e, w = bf(rng, T, 8, D), torch.from_numpy(rng.random((T, 8)).astype(np.float32))
    hd = h.cuda()
    q, s = snr.moe_combine_boundary_fp8(hd, e.cuda(), w.cuda(), pw.cuda(), qw.cuda(), 20)
    snr.sync_status()
    same_bytes(q, f32(oracle.moe_boundary(h, e, w, pw, qw, 20, 1e-6)[1]))


def test_activation():
    F = 640
    x = torch.ones(4, 2 * F)
    x[:, F + 1:F + 128:2] = -1e-9      # beside 1: round to -0, and to 0 where even
    x[:, F + 2:F + 128:2] = 1e-9
    x[:, 128:256] = -0.0               # zeros of both signs
    x[0, F + 128:F + 256] = -3.0
    x[:, 256 + 77] = float("inf")
    x[:, F + 384 + 9] = float("nan")
    x[:, 512:640] = -95.0              # e^-g overflows: zeros
    x = x.to(torch.bfloat16).cuda()
    q, s = snr.swiglu_fp8(x)
    snr.sync_status()
    raw = q.view(torch.uint8)
    assert (raw[:, 0] == 0x7E).all() and (raw[:, 1:128:2] == 0x80).all() and (raw[:, 2:128:2] == 0).all()
    assert not raw[:, 128:].any()
    assert (s[:, 1] == 0).all() and s[:, 2].isposinf().all() and s[:, 3].isnan().all() and (s[:, 4] == 0).all()
