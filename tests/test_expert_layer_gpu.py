"""The calls around the experts one after another, as a decoder layer makes them, and its training step."""
from __future__ import annotations

import pytest
import torch

import sandwich_norm_residual_gb300 as snr
from sandwich_norm_residual_gb300 import build

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn
E, TOPK = 256, 8


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    snr.library()


def rand(g, *s, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(s, generator=g, device="cuda") * scale).to(dtype)


def weights(g, N, K):
    """E4M3 channels with a scale for each 128 by 128, of a size that keeps the outputs near 1."""
    bn, bk = -(-N // 128), -(-K // 128)
    w = torch.nn.functional.pad(torch.randn(E, N, K, generator=g, device="cuda"), (0, bk * 128 - K, 0, bn * 128 - N))
    v = w.view(E, bn, 128, bk, 128)
    s = v.abs().amax((2, 4)) / 448
    q = (v / s[:, :, None, :, None]).clamp(-448, 448).to(FP8).view(E, bn * 128, bk * 128)
    return q[:, :N, :K].contiguous(), s / K ** 0.5


def dequantised(q, s):
    """FP8 rows (or an expert's channels) in 64 bits"""
    rows = 1 if s.shape[0] == q.shape[0] else 128
    s = s.repeat_interleave(rows, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]
    return q.double() * s.double()


@pytest.mark.parametrize("T,pad,graph", [(1, 0, False), (1, 0, True), (5, 2, True), (64, 0, True), (300, 17, False), (2000, 100, True)])
def test_an_expert_layer(T, pad, graph):
    """boundary (FP8) -> routing -> sort -> gather -> gate and up -> activation -> down -> combine -> boundary, with
    padded tokens that have no experts; each step against 64 bits on what the step before it wrote."""
    D, F = 1024, 272
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    h, x, pw, qw = rand(g, T, D), rand(g, T, D), 1 + rand(g, D, scale=0.1), 1 + rand(g, D, scale=0.1)
    (w1, s1), (w2, s2) = weights(g, 2 * F, D), weights(g, D, F)
    router = torch.randn(E, D, generator=g, device="cuda") / D ** 0.5
    bias = torch.zeros(E, device="cuda")
    h0 = h.clone()

    def layer(h):
        y, ys = snr.boundary_fused_fp8(h, x, pw, qw, 5)
        logits = (y.float() * ys.repeat_interleave(128, 1)) @ router.t()
        idx, wt = snr.moe_route(logits, bias)
        if pad:
            idx[T - pad:] = -1
        off, slots = snr.moe_sort(idx, E)
        rows, rs = snr.moe_gather(y, slots, scale=ys)
        gu = snr.matmul_fp8_experts(rows, rs, off, w1, s1)
        act, acts = snr.swiglu_fp8(gu, offsets=off)
        out = snr.matmul_fp8_experts(act, acts, off, w2, s2)
        xc = snr.moe_combine(out, slots, wt)
        z = snr.boundary_fused(h, xc, pw, qw, 6)
        return y, ys, idx, wt, off, slots, rows, rs, gu, act, acts, out, xc, z

    if graph:
        layer(h.clone())  # the plain matrix product sets itself up
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg, stream=side):
            res = layer(h)
        for _ in range(2):
            h.copy_(h0)
            cg.replay()
    else:
        res = layer(h)
    snr.sync_status()
    y, ys, idx, wt, off, slots, rows, rs, gu, act, acts, out, xc, z = res
    n = int(off[-1])
    assert n == (T - pad) * TOPK
    token = torch.empty(n, dtype=torch.int64, device="cuda")
    held = slots >= 0
    token[slots[held].long()] = torch.arange(T, device="cuda")[:, None].expand(T, TOPK)[held]
    assert torch.equal(rows.view(torch.uint8)[:n], y.view(torch.uint8)[token]) and torch.equal(rs[:n], ys[token])
    b = off.tolist()
    for e in range(E):
        lo, hi = b[e], b[e + 1]
        if lo == hi:
            continue
        for q, s, w, sw, got in ((rows, rs, w1, s1, gu), (act, acts, w2, s2, out)):
            a, c = dequantised(q.view(torch.uint8)[lo:hi].view(FP8), s[lo:hi]), dequantised(w[e], sw[e])
            ref, size = a @ c.t(), a.abs() @ c.abs().t()
            # a rounding to BF16, the scales' products, the matrix unit's sums (84 2^-24 of a block's size, as
            # derived for the products alone), those of the blocks and up to eight shares: (blocks + 93) 2^-24
            tol = 2.0 ** -8 * ref.abs() + (8 + 93) * 2.0 ** -24 * 1.01 * size
            assert ((got[lo:hi].double() - ref).abs() <= tol).all()
    gate, up = gu[:n, :F].double(), gu[:n, F:].double()
    v = gate * torch.sigmoid(gate) * up
    # half a step of E4M3 around a value whose scale and size are exact to 2^-19: 2^-4 of it, or 2^-10 of the scale
    sc = acts[:n].repeat_interleave(128, 1)[:, :F].double()
    assert ((dequantised(act.view(torch.uint8)[:n].view(FP8), acts[:n]) - v).abs()
            <= torch.maximum(2.0 ** -4 * v.abs(), 2.0 ** -10 * sc) * 1.001).all()
    parts = torch.where(held[:, :, None], out.double()[slots.clamp(min=0).long()] * wt.double()[:, :, None], 0.0)
    assert ((xc.double() - parts.sum(1)).abs() <= 2.0 ** -8 * parts.sum(1).abs() + 9 * 2.0 ** -24 * parts.abs().sum(1)).all()
    assert not xc[T - pad:].any()
    # the boundary behind it: combined in one call, the same bits
    h2 = h0.clone()
    snr.boundary_fused(h2, x, pw, qw, 5)
    full = torch.where(held[:, :, None], out[slots.clamp(min=0).long()], torch.zeros((), dtype=out.dtype, device="cuda"))
    z2 = snr.moe_combine_boundary(h2, full, torch.where(held, wt, 0.0), pw, qw, 6)
    assert torch.equal(h, h2) and torch.equal(z, z2)


def test_a_training_step_of_the_layer_around_linear_experts():
    """Gradients of gather -> expert (a matrix each) -> combine for tokens, routing weights and experts, against
    PyTorch's own of the same layer in 64 bits."""
    T, D, K, n_exp = 200, 64, 4, 16
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    x, dz = rand(g, T, D, dtype=torch.float32), rand(g, T, D, dtype=torch.float32)
    w = torch.rand(T, K, generator=g, device="cuda")
    mats = rand(g, n_exp, D, D, dtype=torch.float32, scale=D ** -0.5)
    idx = torch.topk(torch.rand(T, n_exp, generator=g, device="cuda"), K).indices.to(torch.int32)
    idx[3, 1] = -1
    idx[-5:] = -1
    off, slots = snr.moe_sort(idx, n_exp)
    b = off.tolist()
    rows = snr.moe_gather(x, slots, out=torch.zeros(T * K, D, device="cuda"))
    out = torch.zeros_like(rows)
    for e in range(n_exp):
        out[b[e]:b[e + 1]] = rows[b[e]:b[e + 1]] @ mats[e]
    z = snr.moe_combine(out, slots, w)
    dout, dw = snr.moe_combine_backward(dz, out, slots, w, drows=torch.zeros_like(out))
    drows, dmats = torch.zeros_like(rows), torch.zeros_like(mats)
    for e in range(n_exp):
        s = slice(b[e], b[e + 1])
        drows[s], dmats[e] = dout[s] @ mats[e].t(), rows[s].t() @ dout[s]
    dx = snr.moe_gather_backward(drows, slots)
    snr.sync_status()

    X, W, M = (t.double().requires_grad_() for t in (x, w, mats))
    one = torch.nn.functional.one_hot(idx.clamp(min=0).long(), n_exp) * (idx >= 0)[:, :, None]
    Z = torch.einsum("tk,tke,td,edf->tf", W, one.double(), X, M)
    (Z * dz.double()).sum().backward()
    for got, ref in ((z, Z), (dx, X.grad), (dw, W.grad), (dmats, M.grad)):
        # a handful of FP32 sums of at most 200 products of size about 1 each: far below 1e-4
        assert (got.double() - ref).abs().max() <= 1e-4 * (1 + ref.abs().max())


@pytest.mark.parametrize("call", ["sort", "gather", "combine", "product", "activation", "boundary"])
def test_operands_made_on_another_stream(call):
    """Calls run on the stream that they are given, behind what is queued there."""
    T, D = 512, 256
    side = torch.cuda.Stream()
    a = torch.full((4096, 4096), 1.0, device="cuda")
    idx = torch.zeros(T, 4, dtype=torch.int32, device="cuda")
    x = torch.zeros(T, D, device="cuda", dtype=torch.bfloat16)
    q = torch.zeros(T, D, device="cuda").to(FP8)
    # ready before anything is queued on the other stream
    slots = torch.arange(4 * T, dtype=torch.int32, device="cuda").view(T, 4)
    rows, wt = torch.ones(4 * T, D, device="cuda"), torch.ones(T, 4, device="cuda")
    w, sa, sw = torch.ones(64, D, device="cuda").to(FP8), torch.ones(T, 2, device="cuda"), torch.ones(1, 2, device="cuda")
    one = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            a = a @ a * 0  # keeps the stream busy
        idx += 2 + a[0, 0].int()
        x += 1 + a[0, 0].to(torch.bfloat16)
        q.copy_(x)
    if call == "sort":
        off, _ = snr.moe_sort(idx, 4, stream=side)
        side.synchronize()
        assert off.tolist() == [0, 0, 0, 4 * T, 4 * T]
    elif call == "gather":
        out = snr.moe_gather(x, slots, stream=side)
        side.synchronize()
        assert (out == 1).all()
    elif call == "combine":
        out = snr.moe_combine(rows, idx, wt, stream=side)
        side.synchronize()
        assert (out == 4).all()
    elif call == "product":
        out = snr.matmul_fp8(q, sa, w, sw, stream=side)
        side.synchronize()
        assert (out == D).all()
    elif call == "activation":
        y, s = snr.swiglu_fp8(x, stream=side)
        side.synchronize()
        assert (y.float() == 448).all() and torch.allclose(s, torch.full_like(s, 0.7310586 / 448))
    else:
        y, _ = snr.boundary_fused_fp8(x, x, one, one, 1, stream=side)
        side.synchronize()
        assert (y.float() == 448).all()
