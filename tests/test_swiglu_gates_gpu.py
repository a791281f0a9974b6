"""The experts' activation at every gate that BF16 has, among them those far below 0 where 1 / (1 + e^-g) leaves FP32's
normal numbers and those where e^-g overflows: y within the header's bound, read off the scale of blocks that hold one value."""
from __future__ import annotations

import pytest
import torch

import sandwich_norm_residual_gb300 as snr
from sandwich_norm_residual_gb300 import build
from test_fp8_rows_gpu import check_swiglu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    snr.library()


def all_gates():
    """Every finite BF16 number, both zeros among them."""
    bits = torch.arange(65536, dtype=torch.int32)
    bits = bits[(bits & 0x7F80) != 0x7F80]
    return bits.to(torch.int16).view(torch.bfloat16).cuda()


@pytest.mark.parametrize("up", [1.0, -3.0, 1.5 * 2.0 ** 60, 3.3e38, 2.0 ** -40, 2.0 ** -120])
def test_every_gate(up):
    """The scale is RN(|y| / 448) and y is within (8 + 2 |g|) 2^-24 of the formula, with half a step of 2^-149 for silu and for y; 0
    where e^-g is past FP32's largest. The one value of a block is its largest: code 448 with y's sign."""
    g = all_gates()
    n, F = len(g), 16
    x = torch.zeros(n, 2 * F, dtype=torch.bfloat16, device="cuda")
    x[:, 5], x[:, F + 5] = g, up
    q, s = snr.swiglu_fp8(x)
    snr.sync_status()
    gd, ud = g.double(), x[:, F + 5].double()
    y = torch.where(gd < -88.72, 0.0, gd * torch.sigmoid(gd)) * ud
    tol = (8 + 2 * gd.abs()) * 2.0 ** -24 * y.abs() + 2.0 ** -149 * (1 + abs(up))
    got = s[:, 0].double() * 448
    tol = tol + 2.0 ** -24 * got + 448 * 2.0 ** -150  # the scale's own half step
    top = torch.finfo(torch.float32).max
    over, under = y.abs() - tol > top, y.abs() + tol < top
    assert (s[over, 0].isinf()).all()
    bad = under & ~((got - y.abs()).abs() <= tol)
    assert not bad.any(), [(float(a), float(b), float(c)) for a, b, c in zip(g[bad][:8], got[bad][:8], y[bad][:8])]
    code = q.view(torch.uint8)[:, 5].int()
    live = under & (s[:, 0] > 0)  # a largest value below 448 2^-150 has codes too, and the scale 0
    assert (code[live] == 0x7E + 0x80 * (y[live] < 0)).all() and not code[gd == 0].any() and not code[over].any()
    others = q.view(torch.uint8).int()
    others[:, 5] = 0
    assert not others.any()


@pytest.mark.parametrize("lo,hi", [(-88.5, -76.0), (-88.5, -87.5)])
def test_blocks_of_gates_far_below_zero(lo, hi):
    """Whole blocks of such gates, among ordinary ones, with factors that bring y back into range."""
    R, F = 96, 272
    g = torch.Generator(device="cuda")
    g.manual_seed(int(-lo - hi))
    x = torch.randn(R, 2 * F, device="cuda", generator=g)
    x[:, 128:256] = lo + (hi - lo) * torch.rand(R, 128, device="cuda", generator=g)
    x[:, F + 128:F + 256] *= 2.0 ** 90
    x[::3, 7] = -88.0  # one lane's value beside others
    x[1::3, 9] = -89.0
    x = x.to(torch.bfloat16)
    q, s = snr.swiglu_fp8(x)
    snr.sync_status()
    assert not q.view(torch.uint8)[1::3, 9].bitwise_and(127).any()
    x[1::3, 9] = 0.0
    check_swiglu(x, q, s)


def test_every_run_gives_the_same_bits():
    x = (torch.randn(4096, 2 * 2560, device="cuda") * 2).to(torch.bfloat16)
    x[17, 40:90] = -87.5
    q, s = snr.swiglu_fp8(x)
    for _ in range(10):
        q2, s2 = snr.swiglu_fp8(x)
        assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)
