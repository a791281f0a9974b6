"""The balance loss at the ends of its ranges: the sigmoid's stated bound over all logits, gradients
where one factor leaves FP32 although the product does not."""
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


@pytest.mark.parametrize("T", [512, 40000])  # one kernel; records and a second kernel
def test_the_sigmoid_is_within_its_bound_at_every_logit(T):
    """A sequence for every token, of four experts whose other logits are infinite (sigmoid 1) and
    whose one choice is the first expert: the loss is alpha 4 p_0 = p_0 = s / (3 + s).

    In units of 2^-24: the sigmoid's stated 8, of which the sum in the denominator takes s / (3 + s)
    back; the sum itself 2 roundings, the division 1, the product 1, the loss 1: 13 at most."""
    z = np.full((T, 4), np.inf, np.float32)
    z[:, 0] = np.linspace(-87, 88, T).astype(np.float32)
    z[:2, 0] = np.float32(-44.371693), np.float32(-44.526)
    idx = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    off = torch.arange(T + 1, dtype=torch.int32, device="cuda")
    loss, counts = snr.moe_balance_loss(torch.from_numpy(z).cuda(), idx, 0.25, seq_offsets=off)
    snr.sync_status()
    s = sigmoid(z[:, 0])
    want = s / (3 + s)
    err = np.abs(loss.cpu().numpy() - want) / want / U
    assert err.max() <= 13, (z[err.argmax(), 0], err.max())
    assert bool((counts[:, 0] == 1).all()) and int(counts.sum()) == T


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
    # units of 2^-24: s (1 - s) 8 + 15 + 1, one over the sum 8 + 21 + 1, their product 1; the factor 6; the
    # mean 8 + 21 + 30 + 1; the difference and two products 3: 124, relative to the two terms. The loss: p
    # 8 + 8 + 11 + 1, its product 1, the loss 1
    got = dz.cpu().numpy()
    assert np.isfinite(got).all()
    assert np.all(np.abs(got - g * (f - mean)) <= 128 * U * np.abs(g) * (f + mean))
    want = alpha * (f * p).sum(1)
    assert np.all(np.abs(loss.cpu().numpy() - want) <= 32 * U * want)
