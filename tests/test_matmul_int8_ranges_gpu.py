"""The 8-bit integer product at the ends of its ranges, bit for bit."""
from __future__ import annotations

import pytest
import torch

import sandwich_norm_residual_gb300 as snr
from sandwich_norm_residual_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    snr.library()
    yield
    torch.cuda.empty_cache()


@pytest.mark.slow
def test_channels_up_to_the_last_31_bit_number():
    """A last tile whose end is channel 2^31, which is no channel (82 GB of operands)."""
    N, K = 2 ** 31 - 8, 16
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    w = torch.randint(-128, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    sw = torch.rand(N, device="cuda", generator=g) + 0.5
    for M in (1, 9):  # dot products; the tensor cores
        a = torch.randint(-128, 128, (M, K), dtype=torch.int8, device="cuda", generator=g)
        sa = torch.rand(M, device="cuda", generator=g) + 0.5
        out = snr.matmul_int8(a, sa, w, sw)
        snr.sync_status()
        for n in (slice(0, 256), slice(2 ** 30 - 128, 2 ** 30 + 128), slice(N - 512, N)):
            ref = (a.double() @ w[n].double().t()).float() * sa[:, None] * sw[n][None, :]
            assert torch.equal(out[:, n], ref.to(torch.bfloat16)), (M, n)
        del out
