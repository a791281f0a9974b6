"""A call captured into a graph as the first that the process makes of the library: nothing that a
first call sets up may end the capture."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PRELUDE = """
import sys
sys.path.insert(0, {root!r})
import torch
import sandwich_norm_residual_gb300 as snr
T, D = 40, 512
bf = lambda *s: torch.ones(s, dtype=torch.bfloat16, device="cuda")
h, x, w, e, tw = bf(T, D), bf(T, D), bf(D), bf(T, 8, D), torch.full((T, 8), 0.125, device="cuda")
a = torch.ones((200, 2560), dtype=torch.int8, device="cuda")
b = torch.ones((5120, 2560), dtype=torch.int8, device="cuda")
sa, sb = torch.ones(200, device="cuda"), torch.ones(5120, device="cuda")
z = torch.zeros((700, 256), device="cuda")
idx = torch.arange(700 * 8, device="cuda").remainder(256).int().view(700, 8)
counts = torch.full((1, 256), 21, dtype=torch.int32, device="cuda")
one = torch.ones(1, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = {call}
g.replay()
torch.cuda.synchronize()
snr.sync_status()
out = out[0] if isinstance(out, tuple) else out
assert bool(torch.isfinite(out.float()).all())
print("captured")
"""

CALLS = {
    "boundary": "snr.boundary_fused(h, x, w, w, 2)",
    "int8": "snr.boundary_fused_int8(h, x, w, w, 2)",
    "product_shared": "snr.matmul_int8(a[:64], sa[:64], b, sb)",
    "product": "snr.matmul_int8(a, sa, b, sb)",
    "balance": "snr.moe_balance_loss(z, idx, 1.0)",
}


@pytest.mark.parametrize("name", CALLS)
def test_first_call(name):
    from sandwich_norm_residual_gb300 import build
    build.build()
    r = subprocess.run([sys.executable, "-c", PRELUDE.format(root=ROOT, call=CALLS[name])], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout[-500:] + r.stderr[-2000:]
