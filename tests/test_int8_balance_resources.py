"""Register budgets of the int8 boundaries, the int8 product and the balance loss: what keeps the CTAs
on an SM that each is launched for, and what may not spill. Read from ptxas's resource summary; no GPU."""
from __future__ import annotations

import re
import subprocess

import pytest

from sandwich_norm_residual_gb300 import build

REGFILE = 65536


@pytest.fixture(scope="module")
def kernels(tmp_path_factory) -> dict[str, tuple[int, int]]:
    """name: (registers a thread, bytes spilled)"""
    d = tmp_path_factory.mktemp("res")
    procs = [subprocess.Popen([build.nvcc()] + build.flags(True) + ["-c", s, "-o", str(d / f"{i}.o")],
                              stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
             for i, s in enumerate(build.SOURCES)]
    out, cur, spilled = {}, None, 0
    for p in procs:
        text = p.communicate()[0]
        assert p.returncode == 0, text[-2000:]
        for line in text.splitlines():
            m = re.search(r"Compiling entry function '(\w+)'", line)
            if m:
                cur = m.group(1)
            m = re.search(r"(\d+) bytes spill stores, (\d+) bytes spill loads", line)
            if m:
                spilled = int(m.group(1)) + int(m.group(2))
            m = re.search(r"Used (\d+) registers", line)
            if m and cur:
                out[cur] = (int(m.group(1)), spilled)
    names = subprocess.run(["c++filt"] + list(out), capture_output=True, text=True).stdout.split("\n")
    return dict(zip(names, out.values()))


def find(kernels, pattern: str) -> tuple[int, int]:
    hits = [v for k, v in kernels.items() if pattern in k]
    assert len(hits) == 1, (pattern, [k for k in kernels if pattern in k])
    return hits[0]


def ctas_per_sm(regs: int, threads: int) -> int:
    return REGFILE // (-(-regs // 8) * 8 * threads)


@pytest.mark.parametrize("vectors,moe,full", [(v, m, f) for v in range(1, 9) for m in ("false", "true")
                                              for f in ("false", "true") if f == "false" or 2 <= v <= 5])
def test_int8_boundaries_hold_their_rows_in_registers(kernels, vectors, moe, full):
    """Up to 6 vectors a thread: no more than the few words (48 bytes, both ways) that some keep over the
    call of the exact row sum. 7 and 8, which only the widest rows take by themselves, spill parts of a row."""
    regs, spilled = find(kernels, f"boundary_int8_kernel<{vectors}, {moe}, {full}>")
    assert regs <= 128
    if vectors <= 6:
        assert spilled <= 48


def test_dense_int8_boundary_keeps_four_ctas_of_128_threads(kernels):
    assert ctas_per_sm(find(kernels, "boundary_int8_kernel<5, false, true>")[0], 128) >= 4


def test_moe_int8_boundary_keeps_two_ctas_of_320_threads(kernels):
    assert ctas_per_sm(find(kernels, "boundary_int8_kernel<2, true, true>")[0], 320) >= 2


@pytest.mark.parametrize("f32", ["false", "true"])
@pytest.mark.parametrize("tile,warps", [("16, 1", 28), ("32, 1", 28), ("64, 1", 28), ("128, 1", 24), ("256, 2", 24)])
def test_product_tiles_fit_an_sm_without_spills(kernels, tile, warps, f32):
    regs, spilled = find(kernels, f"matmul_int8_tile_kernel<{tile}, {f32}>")
    assert ctas_per_sm(regs, 32 * warps) >= 1 and spilled == 0


@pytest.mark.parametrize("f32", ["false", "true"])
@pytest.mark.parametrize("shape,blocks", [("1, 2, 4", 4), ("2, 2, 4", 3), ("4, 4, 3", 2), ("8, 4, 2", 2)])
def test_few_token_products_keep_their_blocks(kernels, shape, blocks, f32):
    regs, spilled = find(kernels, f"matmul_int8_few_kernel<{shape}, {f32}>")
    assert ctas_per_sm(regs, 256) >= blocks and spilled == 0


@pytest.mark.parametrize("vectors", [1, 2, 4])
@pytest.mark.parametrize("kernel", ["records", "small", "grad"])
def test_balance_kernels_hold_their_rows_in_registers(kernels, kernel, vectors):
    """The records of 512 experts keep two words elsewhere."""
    regs, spilled = find(kernels, f"balance_{kernel}_kernel<{vectors}>")
    assert spilled <= (16 if (kernel, vectors) == ("records", 4) else 0)
    if vectors <= 2 and kernel != "small":  # two blocks of 512 threads an SM, as the split assumes
        assert ctas_per_sm(regs, 512) >= 2
