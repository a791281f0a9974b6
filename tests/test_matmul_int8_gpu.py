"""The 8-bit integer product on the GPU against the integer sum in 64 bits.

Integer sums are exact (no partial sum of these inputs leaves +-2^24 unless a test says so), and
the FP32 products that follow are fixed by the header, so outputs are compared bit for bit."""
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


def inputs(M, N, K, seed, lo=-128, hi=128):
    rng = np.random.default_rng(seed)
    return (rng.integers(lo, hi, (M, K), dtype=np.int8), (rng.random(M) + 0.1).astype(np.float32),
            rng.integers(lo, hi, (N, K), dtype=np.int8), (rng.random(N) * 0.01).astype(np.float32))


def want(a, sa, w, sw):
    acc = (a.astype(np.float64) @ w.astype(np.float64).T)  # exact: below 2^53
    with np.errstate(all="ignore"):
        return (acc.astype(np.float32) * sa[:, None]) * sw[None, :]


def run(a, sa, w, sw, dtype=torch.float32, **kw):
    out = snr.matmul_int8(*(torch.from_numpy(v).cuda() for v in (a, sa, w, sw)), out_dtype=dtype, **kw)
    snr.sync_status()
    return out


def check(ops, dtype=torch.float32, **kw):
    got, ref = run(*ops, dtype=dtype, **kw), torch.from_numpy(want(*ops)).to(dtype)
    assert got.dtype == dtype
    assert torch.equal(got.cpu().view(torch.int32 if dtype == torch.float32 else torch.int16),
                       ref.view(torch.int32 if dtype == torch.float32 else torch.int16))


SHAPES = [
    # one token to a few, odd channels, one step of k, and a k that ends inside every tile
    (1, 1, 16), (1, 129, 144), (2, 7, 5120), (3, 2565, 272), (5, 1000, 2064), (8, 640, 128), (1, 6144, 5120),
    # up to a tile of tokens and one past it
    (9, 200, 160), (16, 384, 1040), (17, 127, 2560), (33, 130, 96), (64, 5120, 1024), (65, 257, 528),
    (100, 2565, 400), (128, 128, 128), (129, 129, 112),
    # several tiles in both directions, ragged in each
    (257, 255, 640), (517, 2565, 2576), (300, 4096, 256), (1000, 777, 336), (2048, 2048, 5120),
    # enough tiles for pairs of CTAs: one ragged wave, and several
    (2100, 2600, 400), (4100, 5000, 144), (2048, 2570, 256), (2500, 3333, 160),
    # whole waves and shared tiles: single CTAs, pairs
    (16, 20480, 1040), (700, 5120, 2560), (1030, 5110, 2064), (150, 300, 20480),
    # fewer channels than a tile of them
    (20, 1, 32), (300, 3, 16), (150, 127, 144),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_shapes(M, N, K, dtype):
    check(inputs(M, N, K, M * 7 + N * 3 + K), dtype)


@pytest.mark.parametrize("M", [1, 4, 64, 300])
def test_long_k(M):
    # 7-bit values: 20480 of them stay far below 2^24 in every partial sum
    check(inputs(M, 260, 20480, M, -60, 61))


@pytest.mark.parametrize("M", [1, 8, 40, 256, 600])
def test_extreme_codes(M):
    # all -128 against all -128 or all 127, at the K where sums still cannot leave 2^24
    K, N = 1024, 300
    a = np.full((M, K), -128, np.int8)
    a[::2] = 127
    w = np.full((N, K), -128, np.int8)
    w[1::3] = 127
    one = np.ones(max(M, N), np.float32)
    check((a, one[:M], w, one[:N]))


@pytest.mark.parametrize("M", [1, 8, 40, 300])
def test_sums_past_the_exact_range(M):
    # every term 127 * 127: at most one FP32 rounding for each of the K terms, and the sum itself below 2^30
    K, N = 20480, 140
    ops = (np.full((M, K), 127, np.int8), np.ones(M, np.float32), np.full((N, K), 127, np.int8),
           np.ones(N, np.float32))
    got = run(*ops).cpu().numpy().astype(np.float64)
    assert np.abs(got / (127.0 * 127.0 * K) - 1).max() <= K * 2.0 ** -24


@pytest.mark.parametrize("M", [2, 70, 520])
def test_zero_and_non_finite_scales(M):
    a, sa, w, sw = inputs(M, 150, 320, 5)
    a[1] = 0
    sa[0], sa[1] = np.nan, np.inf
    sw[3], sw[4] = np.inf, 0
    ref = want(a, sa, w, sw)
    got = run(a, sa, w, sw).cpu().numpy()
    assert np.array_equal(got, ref, equal_nan=True)
    assert np.isnan(got[0]).all() and np.isnan(got[1]).all()


@pytest.mark.parametrize("M,N", [(3, 77), (40, 131), (300, 259)])
def test_output_given_neighbours_stay_and_odd_alignment(M, N):
    a, sa, w, sw = inputs(M, N, 256, 9)
    buf = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[3:3 + M * N].view(M, N)  # a 2-byte aligned output
    # scales at 4-byte offsets
    sa_d = torch.zeros(M + 1, device="cuda")[1:]
    sa_d.copy_(torch.from_numpy(sa))
    got = snr.matmul_int8(torch.from_numpy(a).cuda(), sa_d, torch.from_numpy(w).cuda(),
                          torch.from_numpy(sw).cuda(), out=out)
    snr.sync_status()
    assert got.data_ptr() == out.data_ptr()
    assert torch.equal(out.cpu(), torch.from_numpy(want(a, sa, w, sw)).to(torch.bfloat16))
    assert (buf[:3] == 7).all() and (buf[3 + M * N:] == 7).all()


def test_nothing_to_do():
    z = torch.zeros((0, 64), dtype=torch.int8, device="cuda")
    w = torch.ones((5, 64), dtype=torch.int8, device="cuda")
    assert snr.matmul_int8(z, torch.zeros(0, device="cuda"), w, torch.ones(5, device="cuda")).shape == (0, 5)
    assert snr.matmul_int8(w, torch.ones(5, device="cuda"), z, torch.zeros(0, device="cuda")).shape == (5, 0)


@pytest.mark.parametrize("M,N", [(1, 500), (48, 500), (700, 500), (2048, 5120)])
def test_graph_replay_on_a_side_stream_and_pdl(M, N):
    a, sa, w, sw = inputs(M, N, 1040, 3)
    d = [torch.from_numpy(v).cuda() for v in (a, sa, w, sw)]
    outs = [torch.empty((M, N), device="cuda") for _ in range(3)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        snr.matmul_int8(*d, out=outs[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            for o in outs:  # back to back, each allowed to start while the one before ends
                snr.matmul_int8(*d, out=o, pdl=True)
    b = np.roll(a, 1, 1)
    d[0].copy_(torch.from_numpy(b))
    for o in outs:
        o.fill_(-1)
    torch.cuda.synchronize()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    ref = torch.from_numpy(want(b, sa, w, sw))
    for o in outs:
        assert torch.equal(o.cpu(), ref)


@pytest.mark.parametrize("T", [1, 48, 300])
def test_boundary_then_product_in_a_graph(T):
    """The two calls as a decoder layer makes them, one kernel's int8 rows read by the next."""
    D, N = 1024, 390
    rng = np.random.default_rng(T)
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(torch.bfloat16).cuda()  # noqa: E731
    h, x, pw, qw = bf(T, D), bf(T, D), bf(D), bf(D)
    w = torch.from_numpy(rng.integers(-127, 128, (N, D), dtype=np.int8)).cuda()
    sw = torch.rand(N, device="cuda") * 0.01
    q = torch.empty((T, D), dtype=torch.int8, device="cuda")
    s = torch.empty(T, device="cuda")
    out = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    h0 = h.clone()
    y = snr.boundary_fused(h0, x, pw, qw, 3)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        snr.boundary_fused_int8(h, x, pw, qw, 3, y_int8=q, y_scale=s)
        snr.matmul_int8(q, s, w, sw, out=out, pdl=True)
    g.replay()
    torch.cuda.synchronize()
    snr.sync_status()
    assert torch.equal(h, h0)
    assert torch.equal(out.cpu(), torch.from_numpy(want(q.cpu().numpy(), s.cpu().numpy(), w.cpu().numpy(),
                                                        sw.cpu().numpy())).to(torch.bfloat16))
    # against the product with the BF16 y: each y is at most half a step s off (and FP32 roundings of 2^-20 s),
    # so a sum is off by at most (1/2 + 2^-16) s sum|w|; then the output's own half step
    full = y.double().cpu() @ (w.double() * sw.double()[:, None]).cpu().t()
    lim = (0.5 + 2.0 ** -16) * s.double().cpu()[:, None] * (w.double().abs().sum(1) * sw.double()).cpu()[None, :]
    assert ((out.double().cpu() - full).abs() <= lim + 2.0 ** -8 * (full.abs() + lim)).all()


@pytest.mark.parametrize("M,N,K", [(40, 200, 1024), (100, 5120, 2560), (2048, 2560, 640)])
def test_waits_run_out_and_the_next_call_is_whole(M, N, K):
    a, sa, w, sw = inputs(M, N, K, 4)
    d = [torch.from_numpy(v).cuda() for v in (a, sa, w, sw)]
    out = torch.zeros((M, N), device="cuda")
    nb = _lib.load().beam_matmul_int8_workspace(M, N, K)
    ws = torch.empty(max(nb, 16), dtype=torch.uint8, device="cuda")
    st = _lib.load().beam_matmul_int8(torch.cuda.current_stream().cuda_stream or None, *(t.data_ptr() for t in d), M,
                                      N, K, _lib.BEAM_OUT_FP32, out.data_ptr(), ws.data_ptr(), nb,
                                      _lib.BEAM_OPT_TEST_WAIT_TIMEOUT)
    assert st == _lib.BEAM_OK
    with pytest.raises(snr.BeamError) as e:
        snr.sync_status()
    assert e.value.status == _lib.BEAM_ERR_TIMEOUT
    check((a, sa, w, sw))


def test_two_streams_at_once():
    """Products of every kernel in flight on two streams, each with its own workspace."""
    shapes = [(1, 700, 2048), (30, 1500, 4096), (64, 2000, 2048), (200, 1000, 2048), (2048, 2560, 512)]
    jobs = []
    for i, s in enumerate(shapes):
        ops = inputs(*s, i)
        jobs.append(([torch.from_numpy(v).cuda() for v in ops], torch.from_numpy(want(*ops))))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for r in range(10):
        for k, st in enumerate(streams):
            for j in range(len(jobs)):
                d, ref = jobs[(j + k * 2 + r) % len(jobs)]
                with torch.cuda.stream(st):
                    outs.append((snr.matmul_int8(*d, out_dtype=torch.float32), ref))
    torch.cuda.synchronize()
    snr.sync_status()
    for got, ref in outs:
        assert torch.equal(got.cpu(), ref)


@pytest.mark.slow
@pytest.mark.parametrize("M,N,K", [(66000, 33000, 16), (70000, 130, 65536), (20, 70000, 65536)])
def test_operands_and_results_past_32_bits(M, N, K):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    a = torch.randint(-5, 6, (M, K), dtype=torch.int8, device="cuda", generator=g)
    w = torch.randint(-5, 6, (N, K), dtype=torch.int8, device="cuda", generator=g)
    sa, sw = torch.rand(M, device="cuda") + 0.5, torch.rand(N, device="cuda") + 0.5
    out = snr.matmul_int8(a, sa, w, sw)
    snr.sync_status()
    for m in (slice(0, 64), slice(M // 2, M // 2 + 64), slice(M - 64, M)):
        for n in (slice(0, 64), slice(N - 64, N)):
            ref = (a[m].double() @ w[n].double().t()).float() * sa[m][:, None] * sw[n][None, :]
            assert torch.equal(out[m, n], ref.to(torch.bfloat16))


def test_a_timeline_of_boundary_product_norm_and_routing():
    """An int8 decoder layer's front half: boundary, query and key projections, per-head norm; then the
    router's FP32 logits from the same int8 rows, routing, the balance of its choices, and the int8
    combine of the experts' outputs."""
    T, D = 48, 1024
    rng = np.random.default_rng(0)
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(torch.bfloat16).cuda()  # noqa: E731
    i8 = lambda *s: torch.from_numpy(rng.integers(-127, 128, s, dtype=np.int8)).cuda()  # noqa: E731
    h, x, pw, qw = bf(T, D), bf(T, D), bf(D), bf(D)
    y, s = snr.boundary_fused_int8(h, x, pw, qw, 5)
    wq, wk, wr = i8(8 * 128, D), i8(2 * 128, D), i8(256, D)
    sq, sk, sr = (torch.full((w.shape[0],), 1e-3, device="cuda") for w in (wq, wk, wr))
    q = snr.matmul_int8(y, s, wq, sq).view(T, 8, 128)
    k = snr.matmul_int8(y, s, wk, sk).view(T, 2, 128)
    logits = snr.matmul_int8(y, s, wr, sr, out_dtype=torch.float32)
    q0 = q.clone()
    one = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    snr.qk_norm(q, k, one, one, torch.arange(T, dtype=torch.int32, device="cuda"), mode="ssmax")
    idx, wts = snr.moe_route(logits, torch.zeros(256, device="cuda"))
    loss, counts = snr.moe_balance_loss(logits, idx, 0.01)
    e = bf(T, 8, D)
    y2, s2 = snr.moe_combine_boundary_int8(h, e, wts, pw, qw, 6)
    snr.sync_status()
    yn, sn = y.cpu().numpy(), s.cpu().numpy()
    for got, w, sw in ((q0.view(T, -1), wq, sq), (logits, wr, sr)):
        ref = torch.from_numpy(want(yn, sn, w.cpu().numpy(), sw.cpu().numpy()))
        assert torch.equal(got.cpu(), ref.to(got.dtype))
    assert int(counts.sum()) == 8 * T and torch.isfinite(loss).all()
    assert int(y2.abs().amax()) == 127 and torch.isfinite(s2).all()
