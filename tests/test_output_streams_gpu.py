"""A call on a side stream makes its outputs while the current stream still has work queued on memory
that it has freed: the outputs may not lie there."""
from __future__ import annotations

import pytest
import torch

import sandwich_norm_residual_gb300 as snr
from sandwich_norm_residual_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def operands():
    build.build()
    snr.library()
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    T, D, N, E = 600, 1024, 640, 256
    bf = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    h, x, w, e = bf(T, D), bf(T, D), bf(D), bf(T, 8, D)
    tw = torch.rand((T, 8), device="cuda", generator=g)
    a = torch.randint(-127, 128, (T, D), dtype=torch.int8, device="cuda", generator=g)
    b = torch.randint(-127, 128, (N, D), dtype=torch.int8, device="cuda", generator=g)
    sa, sb = torch.rand(T, device="cuda", generator=g), torch.rand(N, device="cuda", generator=g)
    z = torch.randn((T, E), device="cuda", generator=g)
    idx, _ = snr.moe_route(z, z[0])
    _, counts = snr.moe_balance_loss(z, idx, 1.0)
    one = torch.ones(1, device="cuda")
    hs = [h.clone() for _ in range(8)]  # each boundary changes its own
    return {
        "boundary": lambda **k: (snr.boundary_fused(hs.pop(), x, w, w, 2, **k),),
        "int8": lambda **k: snr.boundary_fused_int8(hs.pop(), x, w, w, 2, **k),
        "moe_int8": lambda **k: snr.moe_combine_boundary_int8(hs.pop(), e, tw, w, w, 2, **k),
        "product": lambda **k: (snr.matmul_int8(a, sa, b, sb, **k),),
        "loss": lambda **k: snr.moe_balance_loss(z, idx, 1.0, **k),
        "gradient": lambda **k: (snr.moe_balance_loss_backward(one, z, counts, 8, 1.0, **k),),
    }


@pytest.mark.parametrize("name", ["boundary", "int8", "moe_int8", "product", "loss", "gradient"])
def test_outputs_stay_clear_of_memory_the_current_stream_still_writes(operands, name):
    call, side = operands[name], torch.cuda.Stream()
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
        assert torch.equal(a, b)
