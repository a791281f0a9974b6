"""The FP8 calls and those around the experts where streams and captures meet: outputs made on a side stream
while the current one still writes memory that it has freed, and a capture as the first call of a process."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

import sandwich_norm_residual_gb300 as snr
from sandwich_norm_residual_gb300 import build

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
T, D, E = 600, 1024, 8


@pytest.fixture(scope="module")
def calls():
    build.build()
    snr.library()
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    bf = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    h, x, w, e = bf(T, D), bf(T, D), bf(D), bf(T, 8, D)
    tw = torch.rand((T, 8), device="cuda", generator=g)
    w8 = torch.randn((E, 640, D), device="cuda", generator=g).to(torch.float8_e4m3fn)
    sw = torch.rand((E, 5, D // 128), device="cuda", generator=g)
    idx = torch.randint(0, E, (T, 8), device="cuda", generator=g, dtype=torch.int32)
    off, slots = snr.moe_sort(idx, E)
    a, sa = snr.boundary_fused_fp8(h.clone(), x, w, w, 2)
    rows, rs = snr.moe_gather(a, slots, sa)
    hs = [h.clone() for _ in range(8)]  # each boundary changes its own
    return {
        "boundary": lambda **k: snr.boundary_fused_fp8(hs.pop(), x, w, w, 2, **k),
        "moe": lambda **k: snr.moe_combine_boundary_fp8(hs.pop(), e, tw, w, w, 2, **k),
        "product": lambda **k: (snr.matmul_fp8(a, sa, w8[0], sw[0], **k),),
        "single": lambda **k: (snr.matmul_fp8(a[:1], sa[:1], w8[0], sw[0], **k),),
        "experts": lambda **k: (snr.matmul_fp8_experts(rows, rs, off, w8, sw, **k),),
        "swiglu": lambda **k: snr.swiglu_fp8(x, **k),
        "sort": lambda **k: snr.moe_sort(idx, E, **k),
        "gather": lambda **k: snr.moe_gather(a, slots, sa, **k),
        "combine": lambda **k: (snr.moe_combine(e.view(-1, D), slots, tw, **k),),
        "gather_backward": lambda **k: (snr.moe_gather_backward(e.view(-1, D), slots, **k),),
        "combine_backward": lambda **k: snr.moe_combine_backward(x, e.view(-1, D), slots, tw, **k),
    }


@pytest.mark.parametrize("name", ["boundary", "moe", "product", "single", "experts", "swiglu", "sort", "gather",
                                  "combine", "gather_backward", "combine_backward"])
def test_outputs_stay_clear_of_memory_the_current_stream_still_writes(calls, name):
    call, side = calls[name], torch.cuda.Stream()
    want = call()
    torch.cuda.synchronize()
    stale = [torch.empty_like(t) for t in want]
    torch.cuda._sleep(20_000_000)  # about 10 ms
    for t in stale:
        t.fill_(7)
    freed = {t.data_ptr() for t in stale}
    del stale, t
    got = call(stream=side)
    assert not freed & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    snr.sync_status()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


PRELUDE = """
import sys
sys.path.insert(0, {root!r})
import torch
import sandwich_norm_residual_gb300 as snr
T, D, E = 1000, 512, 16
bf = lambda *s: torch.ones(s, dtype=torch.bfloat16, device="cuda")
h, x, w, rows = bf(T, D), bf(T, D), bf(D), bf(T * 8, D)
tw = torch.full((T, 8), 0.125, device="cuda")
a = torch.ones((T, D), device="cuda").to(torch.float8_e4m3fn)
b = torch.ones((E, 5120, D), device="cuda").to(torch.float8_e4m3fn)
sa, sb = torch.ones((T, 4), device="cuda"), torch.ones((E, 40, 4), device="cuda")
idx = torch.arange(T * 8, device="cuda").remainder(E).int().view(T, 8)
slots = torch.arange(T * 8, device="cuda").int().view(T, 8)
off = torch.arange(E + 1, device="cuda").int() * (T // E)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = {call}
g.replay()
torch.cuda.synchronize()
snr.sync_status()
out = out[0] if isinstance(out, tuple) else out
assert bool(torch.isfinite(out[:T // E * E].float()).all())
print("captured")
"""

FIRST = {
    "boundary": "snr.boundary_fused_fp8(h, x, w, w, 2)",
    "product_single": "snr.matmul_fp8(a[:1], sa[:1], b[0], sb[0])",
    "product_few_shared": "snr.matmul_fp8(a[:40], sa[:40], b[0], sb[0])",
    "product_many": "snr.matmul_fp8(a, sa, b[0], sb[0])",
    "experts": "snr.matmul_fp8_experts(a, sa, off, b, sb)",
    "swiglu": "snr.swiglu_fp8(x)",
    "sort": "snr.moe_sort(idx, E)",
    "gather": "snr.moe_gather(a, slots, sa)",
    "combine": "snr.moe_combine(rows, slots, tw)",
    "combine_backward": "snr.moe_combine_backward(x, rows, slots, tw)",
}


@pytest.mark.parametrize("name", FIRST)
def test_a_capture_as_the_first_call(name):
    build.build()
    r = subprocess.run([sys.executable, "-c", PRELUDE.format(root=ROOT, call=FIRST[name])], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout[-500:] + r.stderr[-2000:]
