"""Sizes that do not fit the 32 bits of the C calls are refused by the binding
(ctypes would cut them: 2^32 + 64 channels would be 64). Tensors without memory
stand for those on the GPU; no call gets as far as the library."""
from __future__ import annotations

import pytest
import torch

BIG = 2 ** 32  # cut to 32 bits it is gone


@pytest.fixture
def tl(monkeypatch):
    import ternary_weight_linear_amd as tl
    tl.lib()
    monkeypatch.setattr(tl, "_on_gpu", lambda t, name: t.device)
    monkeypatch.setattr(tl, "_dev", lambda t, *a, **kw: t)
    monkeypatch.setattr(tl, "_stream", lambda stream: 0)
    return tl


def made(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")


def bf16(*shape):
    return made(*shape, dtype=torch.bfloat16)


def batch(tl, seqs=1):
    i = torch.int32
    return tl.StateBatch(made(seqs + 1, dtype=i), made(seqs, dtype=i), made(seqs, dtype=i), max_q=4)


@pytest.mark.parametrize("rows,ch,slots", [(BIG + 5, 8, 1), (5, BIG + 8, 1), (5, 8, BIG + 1)])
def test_conv(tl, rows, ch, slots):
    with pytest.raises(ValueError, match="32 bits"):
        tl.causal_conv(made(rows, ch), made(ch, 4), made(slots, 3, ch), batch(tl))


@pytest.mark.parametrize("rows,heads,dim,groups,n,slots", [
    (BIG + 5, 4, 64, 2, 64, 1), (5, BIG + 4, 64, 2, 64, 1), (5, 4, BIG + 64, 2, 64, 1), (5, 4, 64, BIG + 2, 64, 1),
    (5, 4, 64, 2, BIG + 64, 1), (5, 4, 64, 2, 64, BIG + 1)])
def test_scan(tl, rows, heads, dim, groups, n, slots):
    b = bf16(rows, groups, n)
    for workspace in (None, made(64, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="32 bits"):
            tl.scan(bf16(rows, heads, dim), b, b, made(rows, heads), made(heads), made(slots, heads, n, dim), batch(tl),
                    out=bf16(rows, heads, dim), workspace=workspace)


@pytest.mark.parametrize("T,K,group", [(BIG + 3, 64, None), (3, BIG + 64, 64), (3, BIG + 64, None), (3, 64, BIG + 64),
                                       (3, 64, 64 - BIG)])
def test_gated_norm(tl, T, K, group):
    x, w = bf16(T, K), made(K)
    for call in (tl.rmsnorm_gated, tl.rmsnorm_gated_s8):
        with pytest.raises(ValueError, match="32 bits"):
            call(x, x, w, group=group)


@pytest.mark.parametrize("T,K", [(BIG + 3, 64), (3, BIG + 64)])
def test_norms_with_a_residual(tl, T, K):
    x, w = bf16(T, K), made(K)
    for call in (tl.rmsnorm_post, tl.rmsnorm_post_s8):
        with pytest.raises(ValueError, match="32 bits"):
            call(x, w, x, w)
    with pytest.raises(ValueError, match="32 bits"):
        tl.rmsnorm_post(x, w, x)
    for call in (tl.rmsnorm, tl.rmsnorm_s8):
        with pytest.raises(ValueError, match="32 bits"):
            call(x, w)


def test_batches_and_positions(tl):
    i = torch.int32
    with pytest.raises(ValueError, match="32 bits"):
        batch(tl, BIG + 2)
    for seqs, width in ((BIG + 2, 1), (2, BIG + 1)):
        with pytest.raises(ValueError, match="32 bits"):
            tl.KVBatch(made(seqs + 1, dtype=i), made(seqs, dtype=i), made(seqs, width, dtype=i), max_q=1, max_kv=1)
    for positions, pairs in ((BIG + 9, 1), (9, BIG + 1)):
        with pytest.raises(ValueError, match="32 bits"):
            tl.Rope(made(positions, pairs, 2))
    with pytest.raises(ValueError, match="32 bits"):
        tl.Rope(made(9, 4, 2))._ref(BIG + 1)
