"""Limits of the decoder operators' launches, checked before any HIP call
(pointers are made up)."""
from __future__ import annotations

import pytest

from tests.test_host_decoder import OK_PTR, SHAPE, structs, tl  # noqa: F401 (fixture)


@pytest.mark.parametrize("heads,seqs", [(1024, 8192), (1024, 8193), (1024, 65535), (257, 65535)])
def test_grids_whose_threads_pass_32_bits_are_refused(tl, heads, seqs):  # noqa: F811
    """2 x heads x seqs workgroups of 256 threads, 2^24 and more."""
    L = tl.lib()
    c, b = structs(tl, dict(heads=heads, dim=64), dict(seqs=seqs, max_q=1))
    row = heads * 64
    assert L.tern_kv_append(c, b, 3, OK_PTR, row, OK_PTR, row, None, 0, 0, None, 0, None, None, None) == SHAPE
    assert b"too large" in L.tern_last_error()
    assert L.tern_kv_read(c, b, 3, OK_PTR, OK_PTR, None) == SHAPE
    assert b"too large" in L.tern_last_error()


def test_append_counts_the_queries_workgroups(tl):  # noqa: F811
    c, b = structs(tl, dict(heads=1, dim=256), dict(seqs=1, max_q=1))
    tokens, heads = 1 << 19, 256  # 2^19 x 256 x 32 threads = 2^32
    got = tl.lib().tern_kv_append(c, b, tokens, OK_PTR, 256, OK_PTR, 256, OK_PTR, heads * 256, heads, OK_PTR, 0, None, None,
                                  None)
    assert got == SHAPE


@pytest.mark.parametrize("seqs", [64, 65, 512])
def test_attention_grids_whose_threads_pass_32_bits_are_refused(tl, seqs):  # noqa: F811
    """8 query heads a kv head, 2^19 rows a sequence: 32768 x 8 workgroups a sequence."""
    L = tl.lib()
    c, b = structs(tl, dict(heads=8), dict(seqs=seqs, max_q=1 << 19))
    assert L.tern_kv_attn(c, b, 3, OK_PTR, 64 * 128, 64, 1.0, 0, 0, OK_PTR, None, 0, None) == SHAPE
    assert b"too many" in L.tern_last_error()
