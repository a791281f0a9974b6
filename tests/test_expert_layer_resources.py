"""Register budgets of the FP8 boundaries and products and of the calls around the experts. Read from ptxas's resource
summary; no GPU."""
from __future__ import annotations

import pytest

from test_int8_balance_resources import ctas_per_sm, find, kernels  # noqa: F401  (the summary is a fixture)


@pytest.mark.parametrize("vectors,moe,full", [(v, m, f) for v in range(1, 9) for m in ("false", "true")
                                              for f in ("false", "true") if f == "false" or 2 <= v <= 5])
def test_fp8_boundaries_hold_their_rows_in_registers(kernels, vectors, moe, full):  # noqa: F811
    """As the int8 ones: up to 6 vectors a thread keep no more than a few words elsewhere."""
    regs, spilled = find(kernels, f"boundary_fp8_kernel<{vectors}, {moe}, {full}>")
    assert regs <= 128
    if vectors <= 6:
        assert spilled <= 64


def test_dense_fp8_boundary_keeps_four_ctas_of_128_threads(kernels):  # noqa: F811
    assert ctas_per_sm(find(kernels, "boundary_fp8_kernel<5, false, true>")[0], 128) >= 4


def test_moe_fp8_boundary_keeps_two_ctas_of_320_threads(kernels):  # noqa: F811
    assert ctas_per_sm(find(kernels, "boundary_fp8_kernel<2, true, true>")[0], 320) >= 2


@pytest.mark.parametrize("f32", ["false", "true"])
def test_product_tiles_fit_an_sm(kernels, f32):  # noqa: F811
    regs, spilled = find(kernels, f"matmul_fp8_kernel<true, {f32}>")
    assert ctas_per_sm(regs, 384) >= 1 and spilled == 0
    # the adding warps ask for 216 registers a thread and the others for 72: what 384 threads of 168 have.
    # With fewer the request would never be met.
    regs, spilled = find(kernels, f"matmul_fp8_kernel<false, {f32}>")
    assert regs == 168 and 256 * 216 + 128 * 72 == 384 * 168 and spilled <= 64


@pytest.mark.parametrize("f32", ["false", "true"])
@pytest.mark.parametrize("warps,blocks,eights", [(8, 3, 1), (4, 6, 1), (8, 3, 2)])
def test_products_of_a_few_tokens_keep_their_blocks(kernels, warps, blocks, eights, f32):  # noqa: F811
    regs, spilled = find(kernels, f"matmul_fp8_small_kernel<{warps}, {blocks}, {eights}, {f32}>")
    assert ctas_per_sm(regs, 32 * warps) >= blocks and spilled <= 64


@pytest.mark.parametrize("pattern,regs,spilled", [
    ("moe_combine_kernel<false, 8>", 72, 0), ("moe_combine_kernel<true, 8>", 72, 0),
    ("moe_combine_kernel<false, 4>", 72, 0), ("moe_combine_kernel<true, 4>", 72, 0),
    ("moe_combine_kernel<false, 2>", 102, 0), ("moe_combine_kernel<true, 2>", 102, 0),
    ("moe_combine_backward_kernel<false, 8>", 80, 0), ("moe_combine_backward_kernel<true, 8>", 80, 0),
    ("moe_combine_backward_kernel<false, 2>", 96, 0), ("moe_combine_backward_kernel<true, 2>", 96, 0),
    ("moe_combine_backward_kernel<false, 16>", 128, 0), ("moe_combine_backward_kernel<true, 16>", 128, 0),
    ("moe_gather_kernel<uint4, uint4>", 40, 0), ("moe_gather_kernel<unsigned int, unsigned int>", 40, 0),
    ("moe_place_kernel", 64, 0), ("moe_count_kernel", 32, 0), ("swiglu_fp8_kernel", 32, 0)])
def test_rows_are_moved_with_many_warps(kernels, pattern, regs, spilled):  # noqa: F811
    got = find(kernels, pattern)
    assert got[0] <= regs and got[1] <= spilled
