"""The balance loss at the ends of its ranges: gradients where one factor leaves FP32 although the
product does not."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import sandwich_norm_residual_gb300 as snr
from sandwich_norm_residual_gb300 import build

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    snr.library()


def sigmoid(z):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-z.astype(np.float64)))


@pytest.mark.parametrize("T", [1, 700])
@pytest.mark.parametrize("level", [-87.0, -80.0, -60.0])
def test_a_scaled_gradient_of_very_negative_logits_is_finite(T, level):
    """The reciprocal of the sigmoids' sum is near 2^125 here and a usual loss scale stands beside it;
    the probabilities and the gradient are ordinary numbers."""
    E, K, alpha, scale = 256, 8, 1e-3, 65536.0
    rng = np.random.default_rng(0)
    z = (level + 0.2 * rng.random((T, E))).astype(np.float32)
    idx = np.tile(np.arange(K, dtype=np.int32), (T, 1))
    off = torch.arange(T + 1, dtype=torch.int32, device="cuda")
    zd = torch.from_numpy(z).cuda()
    loss, counts = snr.moe_balance_loss(zd, torch.from_numpy(idx).cuda(), alpha, seq_offsets=off)
    d = torch.full((T,), scale, device="cuda")
    dz = snr.moe_balance_loss_backward(d, zd, counts, K, alpha, seq_offsets=off)
    snr.sync_status()
    s = sigmoid(z)
    p = s / s.sum(1, keepdims=True)
    f = np.zeros((T, E))
    f[:, :K] = E / K
    mean = (p * f).sum(1, keepdims=True)
    g = scale * alpha * p * (1 - s)
    # units of 2^-24: each sigmoid 91 at z = -87 (|z| + 4), the sum's 91 + 21, the division 1, the factor
    # 4, the mean 91 + 91 + 21 + 1, four products: 416, relative to the two terms; the loss without the
    # factor and the products twice the sigmoid and 30
    got = dz.cpu().numpy()
    assert np.isfinite(got).all()
    assert np.all(np.abs(got - g * (f - mean)) <= 416 * U * np.abs(g) * (f + mean))
    want = alpha * (f * p).sum(1)
    assert np.all(np.abs(loss.cpu().numpy() - want) <= 212 * U * want)
