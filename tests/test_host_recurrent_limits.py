"""Sizes of the recurrent block's operators at the limits of a launch, without
a GPU: what a launch cannot hold is refused before any HIP call."""
from __future__ import annotations

import pytest

from tests.test_host_recurrent import NONE, P, SHAPE, batch, conv, scan, tl  # noqa: F401 (fixture)


@pytest.mark.parametrize("type,per", [(0, 4), (1, 8)])
def test_conv_threads_of_a_sequence_fit_31_bits(tl, type, per):  # noqa: F811
    """A thread's number within its sequence has 31 bits; max_q bounds it, however few the rows."""
    ch = 1 << 20
    runs = (1 << 31) // (ch // per)  # of 16 tokens: 2^31 threads
    for max_q in (16 * runs + 1, 16 * runs + 16, min(2 * 16 * runs - 16, 1 << 19)):
        assert conv(tl, batch(tl, seqs=1, max_q=max_q), rows=32, type=type, ch=ch, xs=ch, ys=ch) == SHAPE, max_q
        assert b"too large" in tl.lib().tern_last_error()


@pytest.mark.parametrize("dim,heads,groups,seqs", [
    (128, 128, 128, 32768), (128, 128, 1, 32768), (64, 256, 2, 32768), (32, 512, 1, 32768), (32, 256, 256, 32768)])
def test_prompt_scan_counts_512_threads_a_workgroup(tl, dim, heads, groups, seqs):  # noqa: F811
    """2^23 workgroups, one for every 64 columns of a group's heads, are 2^32 threads; one sequence less fits."""
    def size(**kw):
        return tl.lib().tern_scan_workspace_bytes(batch(tl, **kw), seqs, heads, dim, groups, 64)

    assert size(seqs=seqs, max_q=9) == NONE
    assert b"too large" in tl.lib().tern_last_error()
    assert 0 < size(seqs=seqs - 1, max_q=9) < NONE
    assert scan(tl, batch(tl, seqs=seqs, max_q=9), rows=seqs, heads=heads, dim=dim, groups=groups, n=64, xs=heads * dim,
                bs=groups * 64, cs=groups * 64, dts=heads, ws=P, wb=1 << 62) == SHAPE


def test_token_scan_counts_256_threads_a_workgroup(tl):  # noqa: F811
    """One workgroup a head, whatever its columns; 2^24 are 2^32 threads."""
    for dim in (32, 128):
        assert tl.lib().tern_scan_workspace_bytes(batch(tl, seqs=32768, max_q=8), 6, 512, dim, 1, 64) == NONE
        assert tl.lib().tern_scan_workspace_bytes(batch(tl, seqs=32767, max_q=8), 6, 512, dim, 1, 64) == 0
