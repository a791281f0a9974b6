"""Refusals of the balance loss, in the C ABI (before any CUDA call) and in the binding: no GPU."""
from __future__ import annotations

import pytest
import torch

import sandwich_norm_residual_gb300 as snr
from sandwich_norm_residual_gb300 import _lib, build

A = 0x7F0000000000  # fake device addresses: never dereferenced
REACHED = (_lib.BEAM_ERR_CUDA, _lib.BEAM_ERR_DEVICE)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_forward_argument_errors(lib):
    Z, I, O, L, C, W = (A + (i << 33) for i in range(6))

    def fw(T=1000, E=256, K=8, S=3, alpha=1.0, z=Z, i=I, o=O, ls=L, c=C, w=W, nb=None):
        nb = lib.beam_moe_balance_workspace(T, E, S) if nb is None else nb
        return lib.beam_moe_balance_loss(None, z, i, o, T, E, K, S, alpha, ls, c, w, nb)

    for kw in (dict(T=-1), dict(T=1 << 31), dict(E=0), dict(E=30), dict(E=516), dict(K=0), dict(K=17), dict(S=0),
               dict(S=1 << 31), dict(o=None)):
        assert fw(**kw) == _lib.BEAM_ERR_SHAPE, kw
    assert fw(alpha=float("nan")) == _lib.BEAM_ERR_ARG
    need = lib.beam_moe_balance_workspace(1000, 256, 3)
    assert need > 0 and fw(nb=need - 1) == _lib.BEAM_ERR_ARG
    for name in ("z", "i", "ls", "c", "w"):
        assert fw(**{name: None}) == _lib.BEAM_ERR_NULL
    for kw in (dict(z=Z + 4), dict(i=I + 2), dict(o=O + 2), dict(ls=L + 1), dict(c=C + 4), dict(w=W + 8)):
        assert fw(**kw) == _lib.BEAM_ERR_ALIGN, kw
    for kw in (dict(ls=C), dict(c=Z + 1024), dict(w=I), dict(ls=O + 4), dict(w=C - 16), dict(c=I - 3056)):
        assert fw(**kw) == _lib.BEAM_ERR_ALIAS, kw
    assert fw() in REACHED
    assert fw(o=None, S=1) in REACHED
    assert fw(T=0, z=None, i=None) in REACHED  # the sequences' zeros are still written
    assert fw(T=512, w=None, nb=0) in REACHED


def test_workspace_sizes(lib):
    ws = lib.beam_moe_balance_workspace
    assert ws(100, 255, 1) == -1 and ws(100, 256, 0) == -1 and ws(-1, 256, 1) == -1
    assert ws(0, 256, 2) == 0 and ws(512, 256, 600) == 0  # one kernel, no records
    assert ws(513, 256, 2) > 0
    # one record for each block and for each sequence: 304 blocks, and no more than 1024 tokens in one
    assert ws(100_000, 256, 5) <= (304 + 5) * 256 * 8
    assert ws(1 << 30, 256, 5) == ((1 << 20) + 5) * 256 * 8


def test_backward_argument_errors(lib):
    G, Z, C, O, D = (A + (i << 33) for i in range(5))

    def bw(T=100, E=256, K=8, S=3, alpha=1.0, g=G, z=Z, c=C, o=O, d=D):
        return lib.beam_moe_balance_loss_backward(None, g, z, c, o, T, E, K, S, alpha, d)

    for kw in (dict(T=-1), dict(E=6), dict(K=0), dict(S=0), dict(o=None)):
        assert bw(**kw) == _lib.BEAM_ERR_SHAPE, kw
    assert bw(alpha=float("inf")) == _lib.BEAM_ERR_ARG
    assert bw(T=0, z=None) == _lib.BEAM_OK
    for name in ("g", "z", "c", "d"):
        assert bw(**{name: None}) == _lib.BEAM_ERR_NULL
    for kw in (dict(g=G + 2), dict(z=Z + 8), dict(c=C + 4), dict(d=D + 4), dict(o=O + 1)):
        assert bw(**kw) == _lib.BEAM_ERR_ALIGN, kw
    for kw in (dict(d=Z), dict(d=C - 1024), dict(g=D + 4), dict(o=D)):
        assert bw(**kw) == _lib.BEAM_ERR_ALIAS, kw
    assert bw() in REACHED


def test_binding_checks():
    T, E = 10, 32
    z, i = torch.zeros((T, E)), torch.zeros((T, 4), dtype=torch.int32)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="shape mismatch"):
        snr.moe_balance_loss(z, i[:5].contiguous(), 1.0)
    with pytest.raises(TypeError, match="topk_idx must be"):
        snr.moe_balance_loss(z, i.long(), 1.0)
    with pytest.raises(TypeError, match="seq_offsets must be"):
        snr.moe_balance_loss(z, i, 1.0, seq_offsets=off.long())
    with pytest.raises(ValueError, match="at least two"):
        snr.moe_balance_loss(z, i, 1.0, seq_offsets=off[:1])
    with pytest.raises(ValueError, match="counts must have shape"):
        snr.moe_balance_loss(z, i, 1.0, seq_offsets=off, counts=torch.zeros((3, E), dtype=torch.int32))
    with pytest.raises(ValueError, match="one device"):
        snr.moe_balance_loss(z, i, 1.0, seq_offsets=off.to("meta"))
    with pytest.raises(ValueError, match="CUDA tensors"):
        snr.moe_balance_loss(z, i, 1.0)
    c = torch.zeros((2, E), dtype=torch.int32)
    with pytest.raises(ValueError, match="dloss must have shape"):
        snr.moe_balance_loss_backward(torch.zeros(1), z, c, 4, 1.0, seq_offsets=off)
    with pytest.raises(ValueError, match="counts must have shape"):
        snr.moe_balance_loss_backward(torch.zeros(1), z, c, 4, 1.0)
    with pytest.raises(ValueError, match="dlogits must have shape"):
        snr.moe_balance_loss_backward(torch.zeros(2), z, c, 4, 1.0, seq_offsets=off, dlogits=torch.zeros((T, 4)))
    with pytest.raises(ValueError, match="CUDA tensors"):
        snr.moe_balance_loss_backward(torch.zeros(2), z, c, 4, 1.0, seq_offsets=off)
