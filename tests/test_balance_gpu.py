"""The router's balance loss, its counts and its gradient against the formula in 64 bits.

Tolerances, u = 2^-24: in the kernel's sigmoid the exponent is rounded once (|z| u, at most 88 u
before e leaves FP32), exp2, the addition and the reciprocal add 2 + 1 + 1 u; p adds a sum of up to
512 sigmoids held as 16 a lane and 5 shuffle levels (21 u), whose own errors are those of its largest
terms, and a division (1 u). A sequence's Q adds at most 64 tokens a warp and 16 warps in FP32: 80
roundings of sums of positive terms, each half a unit of the sum so far, 40 u on average over the terms
and 80 u at most for the first. With logits below 20 in magnitude, where sums are large, 20 + 40 + 80 u;
at 88 they are short (5 tokens a warp): 150 u in all, and REL = 1e-5 is 168 u. Gradients also carry the cancellation in counts_e - sum_i counts_i p_i, so
their bound is relative to counts_e + sum_i counts_i p_i."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import sandwich_norm_residual_gb300 as snr
from sandwich_norm_residual_gb300 import build

pytestmark = pytest.mark.gpu
REL = 1e-5


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    snr.library()


def inputs(T, E, K, seed, scale=2.0):
    rng = np.random.default_rng(seed)
    z = (rng.standard_normal((T, E)) * scale).astype(np.float32)
    idx = np.argsort(-(z + rng.standard_normal((T, E))), axis=1)[:, :K].astype(np.int32)
    return z, np.ascontiguousarray(idx)


def want(z, idx, off, alpha, dloss):
    """(loss, counts, dlogits, magnitude of dlogits' two terms) in 64 bits, sequence by sequence."""
    T, E = z.shape
    K, S = idx.shape[1], len(off) - 1
    loss, counts = np.zeros(S), np.zeros((S, E), np.int64)
    dz, mag = np.zeros((T, E)), np.zeros((T, E))
    for s in range(S):
        lo, hi = off[s], off[s + 1]
        n = hi - lo
        if not n:
            continue
        with np.errstate(over="ignore"):
            sg = 1 / (1 + np.exp(-z[lo:hi].astype(np.float64)))
            co = 1 / (1 + np.exp(z[lo:hi].astype(np.float64)))  # 1 - sg, which would cancel for z > 37
        p = sg / sg.sum(1, keepdims=True)
        counts[s] = np.bincount(idx[lo:hi].ravel(), minlength=E)
        f = counts[s] * E / (K * n)
        loss[s] = alpha * (f * p.mean(0)).sum()
        g = dloss[s] * alpha / n * sg * co / sg.sum(1, keepdims=True)
        mean = (p * f).sum(1, keepdims=True)
        dz[lo:hi] = g * (f - mean)
        mag[lo:hi] = np.abs(g) * (f + mean)
    return loss, counts, dz, mag


def gpu(z, idx, off, alpha, dloss, **kw):
    zd, id = torch.from_numpy(z).cuda(), torch.from_numpy(idx).cuda()
    od = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    loss, counts = snr.moe_balance_loss(zd, id, alpha, seq_offsets=od, **kw)
    dz = snr.moe_balance_loss_backward(torch.from_numpy(dloss).cuda(), zd, counts, idx.shape[1], alpha,
                                       seq_offsets=od, **kw)
    snr.sync_status(kw.get("stream"))
    return loss.cpu().numpy(), counts.cpu().numpy(), dz.cpu().numpy()


def check(z, idx, off, alpha, dloss, given=True, **kw):
    loss, counts, dz, mag = want(z, idx, off, alpha, dloss)
    got = gpu(z, idx, off if given else None, alpha, dloss, **kw)
    assert np.array_equal(got[1], counts)
    assert np.all(np.abs(got[0] - loss) <= REL * np.abs(loss))
    # 2^-140: below it FP32 itself has no more digits
    assert np.all(np.abs(got[2] - dz) <= REL * mag + 2.0 ** -140)
    return got


CASES = [(1, 4, 1), (3, 8, 2), (128, 256, 8), (1000, 256, 8), (777, 64, 6), (50, 132, 3), (4099, 160, 16),
         (333, 512, 8), (20, 388, 1), (16384, 256, 8), (512, 256, 4),
         (513, 256, 4), (600, 512, 8), (530, 4, 2)]


@pytest.mark.parametrize("T,E,K", CASES)
def test_one_sequence(T, E, K):
    z, idx = inputs(T, E, K, T + E)
    check(z, idx, [0, T], 0.001, np.array([1.5], np.float32), given=False)


@pytest.mark.parametrize("T,E,K", [(64, 32, 2), (500, 256, 8), (1000, 256, 8), (5000, 128, 4), (40000, 64, 2)])
def test_ragged_sequences_empty_ones_and_padding(T, E, K):
    rng = np.random.default_rng(T)
    z, idx = inputs(T, E, K, T * 3 + E)
    for S in (1, 2, 7, 33):
        cuts = np.sort(rng.integers(T // 16, T - T // 8, S + 1))
        cuts[1:3] = cuts[1]  # an empty sequence
        off = [int(c) for c in cuts]
        # padding on both sides is not read
        zz = z.copy()
        zz[:off[0]] = np.nan
        zz[off[-1]:] = np.inf
        ii = idx.copy()
        ii[:off[0]] = -5
        ii[off[-1]:] = 1 << 30
        got = check(zz, ii, off, 0.5, rng.random(S).astype(np.float32) - 0.3)
        assert (got[2][:off[0]] == 0).all() and (got[2][off[-1]:] == 0).all()


def test_a_sequence_for_every_token_and_many_blocks():
    T, E, K = 3000, 64, 4
    z, idx = inputs(T, E, K, 1)
    check(z, idx, list(range(T + 1)), 1.0, np.linspace(-1, 1, T).astype(np.float32))


def test_equal_runs_give_equal_bits():
    z, idx = inputs(30000, 256, 8, 2)
    off, d = [0, 100, 100, 17000, 30000], np.ones(4, np.float32)
    first = gpu(z, idx, off, 0.1, d)
    for _ in range(3):
        for a, b in zip(first, gpu(z, idx, off, 0.1, d)):
            assert np.array_equal(a, b)


def test_the_same_expert_twice_and_skewed_choices():
    T, E, K = 600, 256, 8
    z, idx = inputs(T, E, K, 3)
    idx[:] = 7
    got = check(z, idx, [0, T], 1.0, np.ones(1, np.float32))
    assert got[1][0, 7] == T * K


def test_extreme_logits():
    T, E, K = 96, 128, 4
    z, idx = inputs(T, E, K, 4, scale=30.0)
    z[3, :5] = np.inf
    z[4, :] = -np.inf          # every sigmoid 0: p = 0, no gradient
    z[5, 10:] = -np.inf
    z[6, :] = 88.0
    z[7, :] = -87.0
    z[8, ::2] = -120.0
    with np.errstate(all="ignore"):
        zz = z.copy()
        zz[4, :] = 0
        loss, counts, dz, mag = want(zz, idx, [0, T], 1.0, np.ones(1, np.float32))
        # row 4 without its share: p = 1/E each
        loss = loss - (counts[0] * E / (K * T) / (E * T)).sum()
        dz[4] = 0
    got = gpu(z, idx, None, 1.0, np.ones(1, np.float32))
    assert np.abs(got[0] - loss) <= REL * loss
    assert np.all(np.abs(got[2] - dz) <= REL * mag + 2.0 ** -126) and (got[2][4] == 0).all()


@pytest.mark.parametrize("T", [300, 3000])
def test_a_nan_stays_in_its_sequence_and_its_row(T):
    E, K = 64, 2
    z, idx = inputs(T, E, K, 5)
    z[120, 9] = np.nan
    loss, counts, dz = gpu(z, idx, [0, 100, 200, T], 1.0, np.ones(3, np.float32))
    assert np.isnan(loss[1]) and np.isfinite(loss[[0, 2]]).all()
    rows = np.isnan(dz).any(1)
    assert rows[120] and rows.sum() == 1 and np.isnan(dz[120]).all()


def test_gradient_against_differences():
    T, E, K = 40, 32, 3
    z, idx = inputs(T, E, K, 6, scale=1.0)
    off, d = [0, 15, 40], np.array([0.7, -1.3], np.float32)
    _, _, dz = gpu(z, idx, off, 2.0, d)
    rng = np.random.default_rng(0)
    for _ in range(20):
        t, e, h = int(rng.integers(T)), int(rng.integers(E)), 1e-4
        up, dn = z.astype(np.float64), z.astype(np.float64)
        up[t, e] += h
        dn[t, e] -= h
        diff = ((want(up, idx, off, 2.0, d)[0] - want(dn, idx, off, 2.0, d)[0]) * d).sum() / (2 * h)
        # central differences: h^2 / 6 of a third derivative below the loss's own size, and 2^-53 loss / h
        assert abs(dz[t, e] - diff) <= 1e-5 * abs(diff) + 1e-8


@pytest.mark.parametrize("T", [140, 700])
def test_ids_and_offsets_out_of_range_are_reported_and_not_counted(T):
    E, K = 64, 2
    z, idx = inputs(T, E, K, 7)
    bad = idx.copy()
    bad[5, 0], bad[6, 1] = E, -1
    zd = torch.from_numpy(z).cuda()
    loss, counts = snr.moe_balance_loss(zd, torch.from_numpy(bad).cuda(), 1.0)
    with pytest.raises(snr.BeamError):
        snr.sync_status()
    ref = np.bincount(idx.ravel(), minlength=E)
    ref[idx[5, 0]] -= 1
    ref[idx[6, 1]] -= 1
    assert np.array_equal(counts.cpu().numpy()[0], ref)
    off = torch.tensor([0, 60, 40, T + 30], dtype=torch.int32, device="cuda")
    snr.moe_balance_loss(zd, torch.from_numpy(idx).cuda(), 1.0, seq_offsets=off)
    with pytest.raises(snr.BeamError):
        snr.sync_status()
    snr.sync_status()  # the word is clear again


def test_no_tokens():
    z = torch.zeros((0, 64), device="cuda")
    i = torch.zeros((0, 4), dtype=torch.int32, device="cuda")
    loss, counts = snr.moe_balance_loss(z, i, 1.0, seq_offsets=torch.zeros(4, dtype=torch.int32, device="cuda"))
    snr.sync_status()
    assert (loss == 0).all() and (counts == 0).all() and counts.shape == (3, 64)
    assert snr.moe_balance_loss_backward(torch.ones(1, device="cuda"), z, counts[:1].contiguous(), 4, 1.0).shape == (0, 64)


def test_two_graphs_and_a_side_stream():
    T, E, K = 2000, 256, 8
    z, idx = inputs(T, E, K, 8)
    zd, ids = torch.from_numpy(z).cuda(), torch.from_numpy(idx).cuda()
    d = torch.ones(1, device="cuda")
    graphs, outs = [], []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for st in streams:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            loss, counts = snr.moe_balance_loss(zd, ids, 0.3)
            outs.append((loss, counts, snr.moe_balance_loss_backward(d, zd, counts, K, 0.3)))
        graphs.append(g)
    z2 = np.ascontiguousarray(z[::-1])
    zd.copy_(torch.from_numpy(z2))
    torch.cuda.synchronize()
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    loss, counts, dz, mag = want(z2, idx, [0, T], 0.3, np.ones(1))
    for o in outs:
        assert np.array_equal(o[1].cpu().numpy(), counts)
        assert abs(o[0].item() - loss[0]) <= REL * loss[0]
        assert np.all(np.abs(o[2].cpu().numpy() - dz) <= REL * mag + 2.0 ** -140)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    check(z, idx, [0, T], 0.3, np.ones(1, np.float32), stream=side)


def test_routing_then_balance():
    """The router's choices straight into the loss, and the counts it returns."""
    T = 700
    rng = np.random.default_rng(9)
    z = (rng.standard_normal((T, 256)) * 2).astype(np.float32)
    zd = torch.from_numpy(z).cuda()
    idx, _ = snr.moe_route(zd, torch.from_numpy((rng.standard_normal(256) * 0.05).astype(np.float32)).cuda())
    loss, counts = snr.moe_balance_loss(zd, idx, 0.01)
    dz = snr.moe_balance_loss_backward(torch.ones(1, device="cuda"), zd, counts, 8, 0.01)
    snr.sync_status()
    ref = want(z, idx.cpu().numpy(), [0, T], 0.01, np.ones(1))
    assert np.array_equal(counts.cpu().numpy(), ref[1]) and int(counts.sum()) == 8 * T
    assert abs(loss.item() - ref[0][0]) <= REL * ref[0][0]
    assert np.all(np.abs(dz.cpu().numpy() - ref[2]) <= REL * ref[3] + 2.0 ** -140)


@pytest.mark.slow
def test_more_logits_than_32_bits_count():
    T, E, K = 8_500_000, 256, 2  # 2.2e9 logits
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    z = torch.randn((T, E), device="cuda", generator=g)
    idx = torch.randint(0, E, (T, K), device="cuda", generator=g, dtype=torch.int32)
    cut = T - 1000
    off = torch.tensor([0, cut, T], dtype=torch.int32, device="cuda")
    loss, counts = snr.moe_balance_loss(z, idx, 1.0, seq_offsets=off)
    d = torch.ones(2, device="cuda")
    dz = snr.moe_balance_loss_backward(d, z, counts, K, 1.0, seq_offsets=off)
    snr.sync_status()
    tail = want(z[cut:].cpu().numpy(), idx[cut:].cpu().numpy(), [0, T - cut], 1.0, np.ones(1))
    assert np.array_equal(counts[1].cpu().numpy(), tail[1][0])
    assert abs(loss[1].item() - tail[0][0]) <= REL * tail[0][0]
    assert np.all(np.abs(dz[cut:].cpu().numpy() - tail[2]) <= REL * tail[3] + 2.0 ** -140)
    assert torch.equal(counts[0], torch.bincount(idx[:cut].reshape(-1), minlength=E).int())
    # 1.0 * sum f P with counts and probabilities near uniform
    assert abs(loss[0].item() - 1.0) < 1e-3
