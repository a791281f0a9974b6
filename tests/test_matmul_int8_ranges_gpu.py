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


def wide_sums(M, N, K, lo, seed=0):
    """Codes whose partial sums grow with k to half of K and then come back to near nothing."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    a = torch.randint(lo, 128, (M, K), device="cuda", generator=g)
    w = torch.randint(lo, 128, (N, K), device="cuda", generator=g)
    w[:, K // 2:] *= -1
    return a, w


# shared tiles of every size; whole ones of single CTAs (19456 channels: one tile an SM) and of pairs
WIDE = [(1, 260, 20480), (8, 260, 65536), (9, 260, 20480), (20, 260, 65536), (64, 260, 65536), (100, 260, 65536),
        (300, 260, 65536), (128, 19456, 20480), (2304, 2048, 20480)]


@pytest.mark.parametrize("M,N,K", WIDE)
def test_sums_of_large_terms_past_the_exact_range_and_back(M, N, K):
    """Terms that are multiples of 2^12: partial sums up to 2^29 are FP32 numbers, so all are exact."""
    a, w = wide_sums(M, N, K, -128)
    a, w = (torch.where(v >= 0, 64, -64) for v in (a.abs() - 32, w))  # a: mostly one sign
    a8, w8 = a.to(torch.int8), w.to(torch.int8)
    one = torch.ones(max(M, N), device="cuda")
    got = snr.matmul_int8(a8, one[:M], w8, one[:N], out_dtype=torch.float32)
    snr.sync_status()
    n = slice(N - 260 if N > 260 else 0, N)
    assert torch.equal(got[:, n].double(), a8.double() @ w8[n].double().t())


@pytest.mark.parametrize("M,N,K", WIDE)
def test_sums_past_the_exact_range_keep_their_stated_bound(M, N, K):
    """Sums to 2^27 and back, of any codes: K 2^-23 sum |a w| at most (one FP32 rounding or cut a term), and
    none for up to 8 tokens."""
    a, w = (v.to(torch.int8) for v in wide_sums(M, N, K, 60, 1))
    one = torch.ones(max(M, N), device="cuda")
    got = snr.matmul_int8(a, one[:M], w, one[:N], out_dtype=torch.float32)
    snr.sync_status()
    n = slice(N - 260 if N > 260 else 0, N)
    ref, size = a.double() @ w[n].double().t(), a.double().abs() @ w[n].double().abs().t()
    err = (got[:, n].double() - ref).abs()
    if M <= 8:
        assert torch.equal(got[:, n], ref.float())
    else:
        assert bool((err <= K * 2.0 ** -23 * size + 2.0 ** -24 * ref.abs()).all())
