"""The balance loss's largest number of sequences, and which sizes one kernel takes: no GPU.

The search for a block's first sequence looks at 32 places a step; with n sequences left, the last is
at most 32 ceil(n / 32), which has to stay a 32-bit number."""
from __future__ import annotations

import pytest

from sandwich_norm_residual_gb300 import _lib, build

A = 0x7F0000000000  # fake device addresses: never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_the_search_stays_within_32_bits():
    n = _lib.BEAM_BALANCE_MAX_SEQUENCES
    step = (n + 31) // 32
    assert n + 31 < 2 ** 31 and 32 * step < 2 ** 31


@pytest.mark.parametrize("S", [_lib.BEAM_BALANCE_MAX_SEQUENCES + 1, 2 ** 31 - 32, 2 ** 31 - 1])
def test_more_sequences_are_refused(lib, S):
    Z, I, O, L, C, W = (A + (i << 36) for i in range(6))
    assert lib.beam_moe_balance_workspace(1000, 4, S) == -1
    assert lib.beam_moe_balance_loss(None, Z, I, O, 1000, 4, 1, S, 1.0, L, C, W, 1 << 40) == _lib.BEAM_ERR_SHAPE
    assert lib.beam_moe_balance_loss_backward(None, L, Z, C, O, 1000, 4, 1, S, 1.0, W) == _lib.BEAM_ERR_SHAPE


def test_the_largest_number_is_taken(lib):
    Z, I, O, L, C, W = (A + (i << 37) for i in range(6))
    S = _lib.BEAM_BALANCE_MAX_SEQUENCES
    assert lib.beam_moe_balance_workspace(1000, 4, S) > S * 32
    assert lib.beam_moe_balance_loss(None, Z, I, O, 1000, 4, 1, S, 1.0, L, C, W, 1 << 40) in (
        _lib.BEAM_ERR_CUDA, _lib.BEAM_ERR_DEVICE)


def test_one_kernel_where_its_blocks_stay_short(lib):
    """One block a sequence, without a workspace: up to 512 tokens, and 384 rows of 256 logits for each sequence."""
    ws = lib.beam_moe_balance_workspace
    for T, E, S in ((384, 256, 1), (192, 512, 1), (512, 64, 1), (512, 256, 2), (512, 512, 3), (0, 4, 1)):
        assert ws(T, E, S) == 0
    for T, E, S in ((385, 256, 1), (193, 512, 1), (512, 256, 1), (512, 512, 2), (513, 4, 600)):
        assert ws(T, E, S) > 0
