"""Tokens sorted by expert and back on the GPU, against plain loops and 64-bit sums.

Tolerances. A combined value is K FP32 multiply-adds and one rounding: within K 2^-24 sum_k |w row| of the 64-bit sum,
BF16 2^-8 of the value more. A weight's gradient is an FP32 sum of D products: D / 128 of them a thread at most
(multiply-adds in two halves), 5 + 3 + 1 additions after: within (D / 128 + 10) 2^-24 sum_j |dx row|."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import sandwich_norm_residual_gb300 as snr
from sandwich_norm_residual_gb300 import _lib, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    snr.library()


def choices(T, K, E, seed, none=0.1, skew=True):
    rng = np.random.default_rng(seed)
    p = rng.random(E) ** (8 if skew else 0)
    idx = rng.choice(E, (T, K), p=p / p.sum()).astype(np.int32)  # an expert may come twice in a row
    idx[rng.random((T, K)) < none] = -1
    if T > 4:
        idx[T // 2] = -1  # a token without any
        idx[-1] = -1      # and padding
    return idx


def sorted_by_hand(idx, E):
    flat = idx.reshape(-1)
    order = [np.nonzero(flat == e)[0] for e in range(E)]
    offsets = np.cumsum([0] + [len(o) for o in order]).astype(np.int32)
    slots = np.full(flat.shape, -1, np.int32)
    for e, o in enumerate(order):
        slots[o] = offsets[e] + np.arange(len(o))
    return offsets, slots.reshape(idx.shape)


def sort(idx, E, **kw):
    off, slots = snr.moe_sort(torch.from_numpy(idx).cuda(), E, **kw)
    snr.sync_status()
    return off, slots


# ---------------------------------------------------------------- sort

@pytest.mark.parametrize("T,K,E", [(1, 1, 1), (1, 8, 256), (4, 8, 256), (7, 3, 5), (64, 8, 256), (333, 16, 512), (512, 8, 256),
                                   (513, 8, 256), (4096, 1, 2), (5000, 7, 31), (16384, 8, 256), (40000, 16, 512),
                                   (131072, 8, 256), (300001, 1, 1)])
def test_sort(T, K, E):
    idx = choices(T, K, E, T + K)
    off, slots = sort(idx, E)
    ref = sorted_by_hand(idx, E)
    assert np.array_equal(off.cpu().numpy(), ref[0]) and np.array_equal(slots.cpu().numpy(), ref[1])


@pytest.mark.parametrize("T", [100, 20000])
def test_sort_of_one_expert_none_and_all_masked(T):
    for value in (0, 3, 6):
        idx = np.full((T, 4), value, np.int32)
        off, slots = sort(idx, 7)
        assert np.array_equal(slots.cpu().numpy().reshape(-1), np.arange(4 * T))
        assert off.tolist() == [0] * (value + 1) + [4 * T] * (7 - value)
    off, slots = sort(np.full((T, 4), -1, np.int32), 7)
    assert off.tolist() == [0] * 8 and bool((slots == -1).all())


def test_sort_of_no_tokens():
    off, slots = snr.moe_sort(torch.empty((0, 8), dtype=torch.int32, device="cuda"), 256)
    snr.sync_status()
    assert off.shape == (257,) and not off.any() and slots.shape == (0, 8)


@pytest.mark.parametrize("T", [10, 3000])
def test_numbers_that_are_no_expert_count_as_none_and_are_reported(T):
    idx = choices(T, 8, 16, 1)
    bad = idx.copy()
    for i, v in enumerate((16, -2, 2 ** 31 - 1, -2 ** 31)):
        idx[i, i], bad[i, i] = -1, v
    off, slots = snr.moe_sort(torch.from_numpy(bad).cuda(), 16)
    with pytest.raises(snr.BeamError) as e:
        snr.sync_status()
    assert e.value.status == _lib.BEAM_ERR_ARG
    ref = sorted_by_hand(idx, 16)
    assert np.array_equal(off.cpu().numpy(), ref[0]) and np.array_equal(slots.cpu().numpy(), ref[1])


# ---------------------------------------------------------------- gather

def rows_of(x, slots, out):
    """out with the tokens' rows at their slots, by hand."""
    ref = out.clone()
    s = slots.reshape(-1).long()
    token = torch.arange(slots.shape[0], device=s.device).repeat_interleave(slots.shape[1])
    ref[s[s >= 0]] = x[token[s >= 0]]
    return ref


@pytest.mark.parametrize("T,K,D,dtype", [
    (1, 1, 4, torch.uint8), (3, 8, 5120, torch.uint8), (4, 8, 5120, torch.bfloat16), (37, 3, 2, torch.float32),
    (64, 8, 136, torch.bfloat16), (1000, 5, 513, torch.float32), (5000, 8, 1000, torch.uint8), (300, 16, 8, torch.int8),
    (16384, 8, 264, torch.bfloat16), (50, 2, 16384, torch.float64)])
def test_gather_copies_every_byte(T, K, D, dtype):
    idx = choices(T, K, 16, T)
    _, slots = sort(idx, 16)
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    bits = lambda n: torch.randint(0, 256, (n, D * torch.empty(0, dtype=dtype).element_size()), dtype=torch.uint8,  # noqa: E731
                                   device="cuda", generator=g)
    x, out = bits(T), bits(T * K + 3)
    ref = rows_of(x, slots, out)
    got = snr.moe_gather(x.view(dtype), slots, out=out.view(dtype))
    snr.sync_status()
    assert torch.equal(got.view(torch.uint8), ref)


@pytest.mark.parametrize("S", [None, 1, 3, 4, 40])
@pytest.mark.parametrize("T", [5, 700])
def test_gather_with_scales(T, S):
    idx = choices(T, 8, 32, T)
    _, slots = sort(idx, 32)
    x = torch.randn(T, 512, device="cuda").to(torch.float8_e4m3fn)
    sc = torch.rand((T,) if S is None else (T, S), device="cuda")
    R = 8 * T
    out = torch.zeros(R, 512, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    osc = torch.full((R, *sc.shape[1:]), -1.0, device="cuda")
    ref, rsc = rows_of(x.view(torch.uint8), slots, out.view(torch.uint8)), rows_of(sc, slots, osc)
    got, gsc = snr.moe_gather(x, slots, scale=sc, out=out, out_scale=osc)
    snr.sync_status()
    assert torch.equal(got.view(torch.uint8), ref) and torch.equal(gsc, rsc)
    new, nsc = snr.moe_gather(x, slots, scale=sc)  # its own buffers: the rows that are held agree
    held = slots[slots >= 0].long()
    assert torch.equal(new.view(torch.uint8)[held], ref[held]) and torch.equal(nsc[held], rsc[held])


def test_gather_at_odd_addresses():
    T, D = 40, 64
    _, slots = sort(choices(T, 4, 8, 0), 8)
    base = torch.randn(T * D + 2, device="cuda").to(torch.bfloat16)
    x = base[2:].view(T, D)  # 4 bytes into an allocation
    buf = torch.zeros(4 * T * D + 2, dtype=torch.bfloat16, device="cuda")
    out = buf[2:].view(4 * T, D)
    ref = rows_of(x, slots, out)
    assert torch.equal(snr.moe_gather(x, slots, out=out), ref) and not buf[:2].any()


def test_a_slot_outside_is_left_out_and_reported():
    x = torch.randn(6, 64, device="cuda")
    slots = torch.tensor([[0, 1], [2, -1], [9, 3], [-7, 4], [2 ** 31 - 1, -2 ** 31], [5, -1]], dtype=torch.int32, device="cuda")
    buf = torch.full((20, 64), 3.0, device="cuda")
    out = buf[5:14]
    w = torch.ones(6, 2, device="cuda")
    for call in (lambda: snr.moe_gather(x, slots, out=out), lambda: snr.moe_gather_backward(out, slots),
                 lambda: snr.moe_combine(out, slots, w), lambda: snr.moe_combine_backward(x, out.clone(), slots, w, drows=out)):
        got = call()
        with pytest.raises(snr.BeamError) as e:
            snr.sync_status()
        assert e.value.status == _lib.BEAM_ERR_ARG
        assert (buf[:5] == 3).all() and (buf[14:] == 3).all()
    dw = got[1]
    assert dw[2, 0] == 0 and dw[3, 0] == 0 and not dw[4].any()


# ---------------------------------------------------------------- combine and gradients

def combined(rows, slots, w):
    """(sum, sum of the sizes) in 64 bits"""
    held = (slots >= 0)[:, :, None]
    r = rows.double()[slots.clamp(min=0).long()]
    if w is not None:
        r = r * w.double()[:, :, None]
    r = torch.where(held, r, torch.zeros_like(r))
    return r.sum(1), r.abs().sum(1)


def check_sum(got, rows, slots, w):
    ref, size = combined(rows, slots, w)
    tol = slots.shape[1] * 2.0 ** -24 * size
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    assert ((got.double() - ref).abs() <= tol).all()
    assert not got[(slots < 0).all(1)].any()


def layer(T, K, E, D, dtype, seed=0):
    idx = choices(T, K, E, seed + T)
    off, slots = sort(idx, E)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    rows = rand(T * K, D).to(dtype)
    rows[int(off[-1]):] = float("nan")  # rows of nobody
    w = rand(T, K)
    w[slots < 0] = float("nan")         # and their weights
    return idx, slots, rows, w, rand(T, D).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K,E,D", [(1, 1, 1, 8), (1, 8, 256, 5120), (5, 3, 4, 24), (64, 8, 256, 5120), (77, 16, 40, 264),
                                     (200, 9, 20, 1032), (3000, 8, 64, 512), (20000, 2, 16, 128), (9, 7, 5, 32768)])
def test_combine_and_its_gradients(T, K, E, D, dtype):
    idx, slots, rows, w, dx = layer(T, K, E, D, dtype)
    got = snr.moe_combine(rows, slots, w)
    back = snr.moe_gather_backward(rows, slots)
    sentinel = torch.full_like(rows, 9.0)
    drows, dw = snr.moe_combine_backward(dx, rows, slots, w, drows=sentinel)
    snr.sync_status()
    assert drows.data_ptr() == sentinel.data_ptr()
    check_sum(got, rows, slots, w)
    check_sum(back, rows, slots, None)
    held = slots >= 0
    s = slots[held].long()
    token = torch.arange(T, device="cuda")[:, None].expand(T, K)[held]
    # one product, rounded to FP32 and then to the rows' type
    ref = (w[held][:, None] * dx.float()[token]).to(dtype)
    assert torch.equal(drows[s], ref)
    free = torch.ones(T * K, dtype=torch.bool, device="cuda")
    free[s] = False
    assert (drows[free] == 9).all()
    prod = dx.double()[token] * rows.double()[s]
    assert ((dw[held].double() - prod.sum(1)).abs() <= (D / 128 + 10) * 2.0 ** -24 * prod.abs().sum(1)).all()
    assert not dw[~held].any()


def test_gradients_against_differences():
    """sum(combine(rows) * dx) grows by drows and dw for small steps of rows and w: it is linear in each, so
    the step may be large and only FP32 rounding is left."""
    T, K, E, D = 40, 4, 9, 64
    idx, slots, rows, w, dx = layer(T, K, E, D, torch.float32, 3)
    rows, w = torch.nan_to_num(rows), torch.nan_to_num(w)
    drows, dw = snr.moe_combine_backward(dx, rows, slots, w, drows=torch.zeros_like(rows))
    step_r, step_w = torch.randn_like(rows), torch.randn_like(w)
    value = lambda r, c: (snr.moe_combine(r, slots, c).double() * dx.double()).sum()  # noqa: E731
    base = value(rows, w)
    size = (rows.abs().double().sum() + step_r.abs().double().sum()) * 4 * w.abs().max() * dx.abs().max()
    assert abs((value(rows + step_r, w) - base) - (drows.double() * step_r.double()).sum()) <= 2.0 ** -20 * size
    assert abs((value(rows, w + step_w) - base) - (dw.double() * step_w.double()).sum()) <= 2.0 ** -20 * size
    # gather: sum(gather(x) * d) grows by its gradient
    x = torch.randn(T, D, device="cuda")
    zeros = torch.zeros(T * K, D, device="cuda")
    d = torch.randn(T * K, D, device="cuda")
    gx = snr.moe_gather_backward(d, slots)
    moved = snr.moe_gather(x, slots, out=zeros.clone())
    assert abs((moved.double() * d.double()).sum() - (x.double() * gx.double()).sum()) <= 2.0 ** -20 * (moved.abs() * d.abs()).double().sum()


def test_combine_is_the_boundarys_combine():
    """combine, then the dense boundary: the bits of the boundary that combines by itself."""
    T, D = 333, 5120
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    idx = torch.topk(torch.rand(T, 256, generator=g, device="cuda"), 8).indices.to(torch.int32)
    off, slots = snr.moe_sort(idx, 256)
    rows, w = rand(8 * T, D), torch.rand(T, 8, generator=g, device="cuda")
    h, pw, qw = rand(T, D), rand(D), rand(D)
    h2 = h.clone()
    y = snr.moe_combine_boundary(h, rows[slots.long()], w, pw, qw, 20)
    y2 = snr.boundary_fused(h2, snr.moe_combine(rows, slots, w), pw, qw, 20)
    snr.sync_status()
    assert torch.equal(h, h2) and torch.equal(y, y2)


def test_infinite_and_nan_rows_stay_with_their_tokens():
    T, K, D = 64, 4, 256
    idx, slots, rows, w, dx = layer(T, K, 8, D, torch.bfloat16, 7)
    s = int(slots[5].max())
    rows[s, 17] = float("inf")
    got = snr.moe_combine(rows, slots, w)
    owner = int((slots == s).any(1).nonzero()[0])
    bad = ~torch.isfinite(got)
    assert bad[owner, 17] and int(bad.sum()) == 1


# ---------------------------------------------------------------- how they are called

def test_every_run_gives_the_same_bits():
    idx, slots, rows, w, dx = layer(5000, 8, 64, 1024, torch.bfloat16, 2)
    first = snr.moe_combine_backward(dx, rows, slots, w, drows=torch.zeros_like(rows))
    for _ in range(5):
        again = snr.moe_combine_backward(dx, rows, slots, w, drows=torch.zeros_like(rows))
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        off, sl = sort(idx, 64)
        assert torch.equal(sl, slots)


def test_a_weight_gradient_does_not_depend_on_the_batch():
    idx, slots, rows, w, dx = layer(300, 8, 64, 1024, torch.bfloat16, 2)
    _, dw = snr.moe_combine_backward(dx, rows, slots, w)
    _, few = snr.moe_combine_backward(dx[:7].contiguous(), rows, slots[:7].contiguous(), w[:7].contiguous())
    assert torch.equal(dw[:7], few)


def test_two_streams_and_a_graph():
    """Sorts with workspaces of their own on two streams at once, and the chain captured and replayed."""
    jobs = [choices(T, 8, 256, T) for T in (300, 20000, 131072)]
    refs = [sorted_by_hand(j, 256) for j in jobs]
    dev = [torch.from_numpy(j).cuda() for j in jobs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for r in range(8):
        for k, st in enumerate(streams):
            i = (r + k) % 3
            with torch.cuda.stream(st):
                outs.append((i, snr.moe_sort(dev[i], 256)))
    torch.cuda.synchronize()
    for i, (off, slots) in outs:
        assert np.array_equal(off.cpu().numpy(), refs[i][0]) and np.array_equal(slots.cpu().numpy(), refs[i][1])

    T, D = 3000, 256
    idx = torch.from_numpy(choices(T, 8, 64, 1)).cuda()
    x, w = torch.randn(T, D, device="cuda"), torch.rand(T, 8, device="cuda")
    rows, back = torch.zeros(8 * T, D, device="cuda"), torch.empty(T, D, device="cuda")
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        off, slots = snr.moe_sort(idx, 64)
        snr.moe_gather(x, slots, out=rows)
        snr.moe_combine(rows, slots, w, out=back)
    new = choices(T, 8, 64, 9)
    idx.copy_(torch.from_numpy(new))
    x.normal_()
    torch.cuda.synchronize()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    snr.sync_status()
    ref = sorted_by_hand(new, 64)
    assert np.array_equal(slots.cpu().numpy(), ref[1])
    check_sum(back, rows, slots, w)
    # every held choice is the token itself: the sum is x times the held weights
    held = torch.where(slots >= 0, w, torch.zeros_like(w)).double().sum(1)
    assert torch.allclose(back.double(), x.double() * held[:, None], rtol=1e-5, atol=1e-5)


@pytest.mark.slow
def test_rows_past_32_bits():
    T, K, D = 70000, 8, 8192
    idx = torch.randint(0, 256, (T, K), dtype=torch.int32, device="cuda")
    off, slots = snr.moe_sort(idx, 256)
    x = torch.arange(T, device="cuda", dtype=torch.int32)[:, None].expand(T, D // 4).contiguous()
    out = torch.full((T * K, D // 4), -1, dtype=torch.int32, device="cuda")  # 4.6 GB
    snr.moe_gather(x, slots, out=out)
    snr.sync_status()
    token = torch.arange(T, device="cuda", dtype=torch.int32).repeat_interleave(K)
    ref = torch.empty(T * K, dtype=torch.int32, device="cuda")
    ref[slots.reshape(-1).long()] = token
    assert torch.equal(out[:, 0], ref) and torch.equal(out[:, -1], ref)
    rows = torch.zeros(T * K, D, dtype=torch.bfloat16, device="cuda")  # 9 GB
    rows[:, 0] = 1
    rows[:, D - 1] = 2
    w = torch.ones(T, K, device="cuda")
    got = snr.moe_combine(rows, slots, w)
    assert (got[:, 0] == 8).all() and (got[:, D - 1] == 16).all() and not got[:, 1:-1].any()
    dx = torch.ones(T, D, dtype=torch.bfloat16, device="cuda")
    _, dw = snr.moe_combine_backward(dx, rows, slots, w, drows=torch.empty_like(rows))
    assert (dw == 3).all()
